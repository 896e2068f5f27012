"""Workspace sizes of the attention to states of another length; no GPU needed."""
import neighborhood_attention_video_gb300 as na
from neighborhood_attention_video_gb300 import build as na_build


def test_sums_of_dq_take_one_gradients_room():
    """Few tokens: dq's pass splits the states, 256 to a split at least, dk and dv's does not.
    Room for one fp32 dq a split and two copies of each row's two statistics is enough."""
    na_build.build()
    for L, S, NH, HD in ((128, 512, 16, 128), (64, 2048, 8, 64), (1, 4096, 32, 16)):
        rows = L * NH
        need = na.na3d_cross_workspace(1, L, S, NH, NH, HD, True)
        assert need <= S // 256 * rows * HD * 4 + 2 * (rows * 8 + 128), (L, S, NH, HD, need)
        assert need > 2 * rows * 8


def test_the_self_test_refuses_what_the_calls_refuse():
    import ctypes
    na_build.build()
    lib, P = na.load_library(), ctypes.c_void_p
    at = [P((1 << 30) + (i << 26)) for i in range(10)]     # never touched
    for sizes, code in (((0, 100, 40, 4, 2, 32), 2), ((2, 100, 40, 4, 3, 32), 2), ((2, 100, 40, 4, 2, 256), 11)):
        assert lib.na3d_cross_selftest_withhold(*at, *sizes, None, None, None) == code
    for i in (0, 1, 2, 3, 4, 6, 7, 8, 9):                  # (without dout it is the forward call)
        assert lib.na3d_cross_selftest_withhold(*at[:i], None, *at[i + 1:], 2, 100, 40, 4, 2, 32, None, None, None) == 1
