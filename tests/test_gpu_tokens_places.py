"""dispatch_tokens on many choices, every row compared with a stable sort's: rows past 2^31 elements, and more chunks of
choices than the GPU has SMs (a chunk has 65,535 at most)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _check(x, idx, E, got):
    rows, offsets, pos = got
    T, k = idx.shape
    on = (idx >= 0) & (idx < E)
    key = torch.where(on, idx, E).flatten()
    order = key.sort(stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device="cuda")
    assert torch.equal(pos.long(), torch.where(on, place.view(T, k), ~place.view(T, k)))
    assert torch.equal(offsets.long(), torch.cat([place.new_zeros(1), torch.bincount(key, minlength=E + 1)[:E].cumsum(0)]))
    live = key[order] < E
    for r in range(0, T * k, 1 << 16):
        at = slice(r, r + (1 << 16))
        want = torch.where(live[at, None], x[order[at] // k], torch.zeros((), dtype=x.dtype, device="cuda"))
        assert torch.equal(rows[at], want)


def test_rows_past_31_bits():
    import sparse_mixture_experts_gemv_gb300 as M
    T, k, E, H = 70000, 8, 64, 4096
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randint(-8, 9, (T, H), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    idx = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    got = M.dispatch_tokens(x, idx, E)
    _check(x, idx, E, got)
    # the sums of the columns: whole numbers, exact in 64 bits
    want = (x.double() * (idx >= 0).sum(1, keepdim=True)).sum(0)
    assert torch.equal(sum(part.sum(0, dtype=torch.float64) for part in got[0].split(1 << 16)), want)


@pytest.mark.parametrize("T,k,E", [(10_100_003, 1, 1000), (1_400_001, 8, 64), (340_000, 31, 1024)])
def test_more_chunks_than_sms(T, k, E):
    import sparse_mixture_experts_gemv_gb300 as M
    assert T * k > 65535 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator("cuda").manual_seed(2)
    x = torch.randint(0, 256, (T, 5), generator=g, device="cuda", dtype=torch.uint8)
    idx = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    idx[T // 3:T // 2] = E // 2   # chunks of one expert
    _check(x, idx, E, M.dispatch_tokens(x, idx, E))
