"""A PoolSet follows its tensors: their memory may be exchanged, their shape may not."""
import pytest
import torch

from paged_kv_decode_cache_gb300 import pa
from test_pages import _built, dev, make_pools, run_fork  # noqa: F401


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_memory_that_was_exchanged_is_used(fp8):
    pools = make_pools(2, 8, 16, 1, 64, fp8, 1)
    held = pa.PoolSet(pools)
    first = [t.clone() for t in pools]
    old = [t.detach() for t in pools]            # the memory of before, kept alive
    others = make_pools(2, 8, 16, 1, 64, fp8, 2)
    want = [t.clone() for t in others]
    pools[0].data = others[0]
    pools[1].set_(others[1])
    pa.pa_blocks_copy(held, dev([[3, 0]]))
    torch.cuda.synchronize()
    for t, w, o, f in zip(pools, want, old, first):
        w[0] = w[3]
        assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))
        assert torch.equal(o.view(torch.uint8), f.view(torch.uint8))   # the old memory is left alone


@pytest.mark.gpu
def test_pools_that_changed_their_shape_are_refused():
    nb = 8
    status, ws = dev([0]), torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    tables, lens, refs = dev([[0, 1]]), dev([20]), dev([1, 1] + [0] * (nb - 2))
    new = [torch.empty(1, 2, dtype=torch.int32, device="cuda"), dev([0]), dev([0] * nb)]
    changes = {
        "smaller": lambda t: t.resize_(4, 16, 1, 64),
        "transposed": lambda t: t.set_(torch.zeros(16, nb, 1, 64, dtype=t.dtype, device="cuda").transpose(0, 1)),
        "gone": lambda t: t.untyped_storage().resize_(0),
    }
    for name, change in changes.items():
        pools = make_pools(2, nb, 16, 1, 64, False, 1)
        held = pa.PoolSet(pools)
        change(pools[1])
        with pytest.raises(ValueError, match="pool"):
            pa.pa_blocks_copy(held, dev([[3, 0]]), status=status)
        with pytest.raises(ValueError, match="pool"):
            pa.pa_sequences_fork(*new, dev([0], torch.int64), tables, lens, refs, dev([0]), held, ws, status=status)
        with pytest.raises(ValueError, match="pool"):
            pa.pa_blocks_compact(new[0], new[2], dev([0] * nb), dev([0]), tables, lens, refs, held, ws, status=status)
    torch.cuda.synchronize()
