"""No GPU: token counts so near 2^31 that the kernels' 32-bit row numbers would
pass it on a last step beyond the end are refused on the host."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(4096)  # never read: every call below fails on the host
MOST = 2 ** 31 - 1 - 2 ** 20
OVER = (MOST + 1, 2 ** 31 - 1)


@pytest.fixture(scope="module")
def lib():
    from linear_attention_sequence_device_gb300 import build, binding
    build.build_library()
    return binding.load()


def calls(lib, T, x):
    ws = (FAKE, 1 << 62)
    seqs = (FAKE, 1)
    return dict(
        conv_fwd=lambda: lib.gdn_ssm_conv_fwd(x, 8, 1, T, 8, FAKE, None, 4, *seqs, None, None, ctypes.c_void_p(8192), 8,
                                              None),
        conv_bwd=lambda: lib.gdn_ssm_conv_bwd(x, 8, FAKE, 8, 1, T, 8, FAKE, None, 4, *seqs, None, None, FAKE, 8, FAKE,
                                              None, None, *ws, None),
        scan_fwd=lambda: lib.gdn_ssm_scan_fwd(x, 8, FAKE, 8, None, 0, FAKE, 1, FAKE, 1, 1, FAKE, None, None, None, *seqs,
                                              T, 8, 1, 1, FAKE, 8, None, None, *ws, None),
        scan_bwd=lambda: lib.gdn_ssm_scan_bwd(x, 8, FAKE, 8, FAKE, 8, None, 0, FAKE, 1, FAKE, 1, 1, FAKE, None, None,
                                              None, FAKE, None, *seqs, T, 8, 1, 1, FAKE, FAKE, None, FAKE, FAKE, FAKE,
                                              None, None, None, *ws, None),
        norm_fwd=lambda: lib.gdn_block_norm_fwd(x, 8, None, 0, 1, FAKE, 1, None, FAKE, None, 1e-6, T, 8, FAKE, FAKE,
                                                None),
        norm_bwd=lambda: lib.gdn_block_norm_bwd(x, None, FAKE, 8, None, 0, 1, FAKE, 1, None, FAKE, None, 1e-6, T, 8,
                                                FAKE, None, FAKE, FAKE, None, None, *ws, None))


NAMES = ("conv_fwd", "conv_bwd", "scan_fwd", "scan_bwd", "norm_fwd", "norm_bwd")


@pytest.mark.parametrize("name", NAMES)
def test_too_many_tokens(lib, name):
    for T in OVER:
        assert calls(lib, T, FAKE)[name]() == 2
        assert b"tokens" in lib.gdn_last_error()
    assert calls(lib, MOST, None)[name]() == 1  # the most is not refused: what is wrong there is the missing array


def test_sizes(lib):
    for size in (lambda T: lib.gdn_ssm_conv_bwd_workspace_size(T, 8, 4), lambda T: lib.gdn_ssm_scan_ckpt_floats(T, 8, 1),
                 lambda T: lib.gdn_ssm_scan_workspace_size(T, 8, 1, 1),
                 lambda T: lib.gdn_ssm_scan_bwd_workspace_size(T, 8, 1, 1), lambda T: lib.gdn_block_norm_bwd_workspace_size(T, 8)):
        assert size(MOST) > 0 and all(size(T) == 0 for T in OVER)
    assert lib.gdn_ssm_scan_ckpt_floats(MOST, 8, 1) == 8 * ((MOST + 7) // 8)


def test_conv_results_over_its_inputs(lib):
    """Strips read rows of their neighbours, so that a result in an input's place would be read as one."""
    other, ws = ctypes.c_void_p(8192), (FAKE, 1 << 62)
    assert lib.gdn_ssm_conv_fwd(FAKE, 8, 1, 100, 8, FAKE, None, 4, FAKE, 1, None, None, FAKE, 8, None) == 1
    assert b"y" in lib.gdn_last_error()
    for dy, x in ((FAKE, other), (other, FAKE)):
        assert lib.gdn_ssm_conv_bwd(dy, 8, x, 8, 1, 100, 8, FAKE, None, 4, FAKE, 1, None, None, FAKE, 8, FAKE, None, None,
                                    *ws, None) == 1
        assert b"dx" in lib.gdn_last_error()
