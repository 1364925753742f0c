"""Sizes that pass a C int are refused by the state space layer's torch entry points,
which hand them to the library as ints (no GPU needed: the tensors have shapes only, and
every call here is refused before anything is read).  The library would see their lowest
32 bits: a cache of 2^32 + 5 rows as one of five, whose other rows are none."""
import pytest
import torch

import recurrent_state_update_amd as rsu


class OnGpu(torch.Tensor):
    """A tensor without data that says it is on a GPU."""
    device = property(lambda self: torch.device("cuda:0"))
    is_cuda = True


def gpu(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="meta").as_subclass(OnGpu)


C, N, MANY = 8, 4, (1 << 32) + 5
I32 = torch.int32
w, x, bc, a = gpu(C, 4), gpu(5, C), gpu(5, N), gpu(C, N)
rows = gpu(5, dtype=I32)


@pytest.mark.parametrize("many", [1 << 31, MANY])
@pytest.mark.parametrize("named", [False, True])
def test_rows_of_a_cache(named, many):
    kw = dict(rows=rows if named else None)
    with torch.no_grad():
        with pytest.raises(ValueError, match=f"{many} rows of states: want fewer"):
            rsu.short_conv_step(x, gpu(many, 3, C), w, **kw)
        with pytest.raises(ValueError, match=f"{many} rows of states: want fewer"):
            rsu.ssm_step(x, x, gpu(many, C, N), a, bc, bc, **kw)


@pytest.mark.parametrize("many", [1 << 31, MANY])
def test_sequences(many):
    cu, none = gpu(many + 1, dtype=I32), (gpu(many, 0, C), gpu(many, 0, N))
    for call in (lambda: rsu.short_conv(x, w, cu_seqlens=cu), lambda: rsu.short_conv(none[0], w),
                 lambda: rsu.ssm_scan(x, x, a, bc, bc, cu_seqlens=cu),
                 lambda: rsu.ssm_scan(none[0], none[0], a, none[1], none[1])):
        with pytest.raises(ValueError, match=f"{many} sequences: want fewer"):
            call()


@pytest.mark.parametrize("many", [1 << 31, MANY])
def test_channels(many):
    with torch.no_grad():
        for call in (lambda: rsu.short_conv(gpu(0, many), gpu(many, 4)),
                     lambda: rsu.short_conv_step(gpu(1, many), gpu(1, 3, many), gpu(many, 4)),
                     lambda: rsu.ssm_scan(gpu(0, many), gpu(0, many), gpu(many, N), gpu(0, N), gpu(0, N)),
                     lambda: rsu.ssm_step(gpu(1, many), gpu(1, many), gpu(1, many, N), gpu(many, N), gpu(1, N), gpu(1, N))):
            with pytest.raises(ValueError, match=f"{many} channels: want fewer"):
                call()
