"""CPU: what the decoder layer's paged step refuses before any of its work.  No test here
launches a kernel."""
import pytest
import torch

from segmented_gather_matmul_amd import build as build_mod
from segmented_gather_matmul_amd import layer as LY
from segmented_gather_matmul_amd import step as S

H, KV, D, T = 4, 2, 64, 8
SHAPE = LY.LlamaShape("case", H * D, 512, H, D, kv_heads=KV)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if build_mod.stale():
        build_mod.build()


def _cache(pages=6, page=8, kv=KV, d=D):
    z = lambda: torch.zeros(pages, page, kv, d, dtype=torch.float16)
    return S.PagedKV(z(), z())


@pytest.fixture(scope="module")
def layer():
    return LY.random_layer(SHAPE, 2, 8, T, torch.Generator().manual_seed(0), device="cpu")


@pytest.mark.parametrize("kw", [dict(page=16), dict(page=4), dict(pages=5), dict(kv=1), dict(kv=4), dict(d=32), dict(d=128)],
                         ids=str)
def test_a_cache_of_another_geometry_is_refused(layer, kw):
    """The operators take the page size, page count and heads from the cache, the slots and
    tables from the step: with others than the step's they would find other cells."""
    step = LY.PagedStep(SHAPE, 2, T, 3, 6, 8, device="cpu")
    hidden = torch.zeros(T, H * D, dtype=torch.float16)
    with pytest.raises(ValueError, match="cache"):
        layer.forward_paged(hidden, _cache(**kw), step, None)
    for fits in (_cache(), _cache(pages=7), step.new_cache(device="cpu")):
        with pytest.raises(ValueError, match="GPU tensor"):       # goes on to the first operator
            layer.forward_paged(hidden, fits, step, None)


def test_a_step_refuses_a_rope_it_has_no_positions_for():
    """A step's rows have one position each (plan.tok_pos), and heads of head_dim columns: refused
    where the step is made, not in a layer after a plan has moved pages."""
    make = lambda rope: LY.PagedStep(SHAPE, 2, T, 3, 6, 8, rope=rope, device="cpu")
    for rope in (None, S.Rope.base(D, device="cpu"), S.Rope.base(D // 2, interleaved=True, device="cpu"),
                 S.Rope.base(D, axis=torch.zeros(D // 2, dtype=torch.int32), device="cpu")):
        assert make(rope).rope is rope
    for rope, msg in ((S.Rope.base(D, axes=2, device="cpu"), "axes"), (S.Rope.base(2 * D, device="cpu"), "columns")):
        with pytest.raises(ValueError, match=msg):
            make(rope)
