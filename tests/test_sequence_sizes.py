"""Buffer sizes of the sequence operators at the ends of what they take (no GPU
needed)."""
import recurrent_state_update_amd as rsu

SHAPE = 2
F32, BF16 = 0, 1
A = [0x7f0000000000 + (i << 40) for i in range(4)]  # aligned, far apart, never dereferenced


def test_gated_norm_workspace_of_refused_sizes():
    """Sizes that the calls refuse have no workspace (their product passed 64
    bits)."""
    big = (1 << 31) - 1
    for rows, H, d in ((big, big, 128), (big, 1 << 20, 16), (1 << 20, 1 << 10, 64)):
        assert rsu.dl_gated_norm(rows, H, d, F32, BF16, A[0], A[1], 0, A[2], 1e-6, A[3], stream=0) == SHAPE
        assert rsu.dl_gated_norm_workspace_bytes(rows, H, d) == 0
    assert rsu.dl_gated_norm_workspace_bytes((1 << 20) - 1, 1 << 7, 64) > 0
