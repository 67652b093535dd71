"""Room in the layer norm gradient's workspace for the blocks that its forms run."""
import pytest

from sampling_gnn_mini_gb300 import binding as sg


# columns, blocks an SM (512 threads an SM with 16 values each, 384 with 24), also of rows
# that are a few values longer than the whole vectors of a form's threads
@pytest.mark.parametrize("dim,per_sm", [(513, 8), (1024, 8), (1025, 8), (1027, 8), (1032, 5), (2048, 4), (2049, 4), (2051, 4), (2060, 3),
                                        (3200, 2), (4096, 2), (4097, 2), (4103, 2), (4104, 2), (4608, 2), (4615, 2), (5000, 1),
                                        (8192, 1), (16384, 1)])
def test_room_for_the_blocks_of_every_form(dim, per_sm):
    blocks = 148 * per_sm // 8 * 8  # (148 SMs when there is no device; a multiple of 8)
    lib = sg.load()
    assert lib.sg_layernorm_bwd_workspace(1 << 20, dim) >= blocks * 2 * dim * 4
    assert lib.sg_layernorm_bwd_workspace(3, dim) < 3 * 2 * (dim + 16) * 4 + 256
