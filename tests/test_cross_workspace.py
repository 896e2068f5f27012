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
