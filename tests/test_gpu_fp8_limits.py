"""GPU tests of the E4M3 and grouped operators at the largest sizes that they take: launches and counts at their
limits, results compared whole on the device, or in part where they have billions of values."""
import pytest

from quantized_expert_ffn_topk_amd import abi

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda"
FP8 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def new(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV)


def test_codes_of_as_many_rows_as_are_taken():
    """2^25 rows of one value: code 448 with its sign, scale |x|/448."""
    T = 1 << 25
    x = torch.randn((T, 1), generator=gen(1), device=DEV).bfloat16()
    x[::1000] = 0
    q, s = new(T, 1, dtype=torch.uint8), new(T, 1, dtype=torch.float32)
    torch.cuda.synchronize()
    abi.moe_quant_fp8(x, abi.DT_BF16, 1, abi.ACT_NONE, T, 1, None, q, 1, s, 1)
    torch.cuda.synchronize()
    v = x.float()
    assert torch.equal(s, v.abs() / torch.full_like(v, 448.0))
    want = torch.where(v == 0, 0, torch.where(v > 0, 0x7e, 0xfe)).to(torch.uint8)
    assert torch.equal(torch.where(v == 0, q & 0x7f, q), want)


def test_codes_of_as_many_blocks_as_are_taken():
    """2^20 rows of 2^14 values, 2^27 blocks in all: rows that repeat 512 ones."""
    T, K, n = 1 << 20, 1 << 14, 512
    few = torch.randn((n, K), generator=gen(2), device=DEV).bfloat16()
    x, q, s = new(T, K, dtype=torch.bfloat16), new(T, K, dtype=torch.uint8), new(T, K // 128, dtype=torch.float32)
    x.view(T // n, n, K).copy_(few)
    qf, sf = new(n, K, dtype=torch.uint8), new(n, K // 128, dtype=torch.float32)
    torch.cuda.synchronize()
    abi.moe_quant_fp8(few, abi.DT_BF16, K, abi.ACT_NONE, n, K, None, qf, K, sf, K // 128)
    abi.moe_quant_fp8(x, abi.DT_BF16, K, abi.ACT_NONE, T, K, None, q, K, s, K // 128)
    torch.cuda.synchronize()
    del x
    assert torch.equal(sf, few.float().view(n, -1, 128).abs().amax(2) / torch.full_like(sf, 448.0))
    for i in range(0, T, 1 << 16):
        assert bool((q[i:i + (1 << 16)].view(-1, n, K) == qf).all()) and bool((s[i:i + (1 << 16)].view(-1, n, K // 128) == sf).all())


# whole numbers of small codes: every sum is exact in fp32, and in bf16 where it is below 2^8
def small_codes(g, n, K):
    return torch.randint(-1, 2, (n, K), generator=g, device=DEV).to(FP8)


def ones(n, K):
    return torch.ones((n, -(-K // 128)), device=DEV)


@pytest.mark.parametrize("T,N,K,pad", [(1 << 20, 1 << 15, 100, 0), (1 << 20, 1 << 15, 9, 0), (1 << 20, 1, 130, 0), (1, 1 << 20, 130, 0),
                                       (33, 1 << 20, 130, 1), (1 << 15, 1 << 20, 4, 0)])
def test_products_of_as_many_results_as_are_taken(T, N, K, pad):
    g = gen(3)
    x, w = small_codes(g, T, K + pad), small_codes(g, N, K + pad)
    y = new(T, N, dtype=torch.bfloat16)
    y.fill_(77)
    s, ws = ones(T, K), ones(-(-N // 128), K)
    torch.cuda.synchronize()
    abi.moe_linear_fp8(x, K + pad, s, s.shape[1], T, w, K + pad, ws, ws.shape[1], None, N, K, y, abi.DT_BF16, N)
    torch.cuda.synchronize()
    xv, wv = x[:, :K].float(), w[:, :K].float().t().contiguous()
    step = max(1, (1 << 29) // N)
    for i in range(0, T, step):
        assert torch.equal(y[i:i + step], (xv[i:i + step] @ wv).bfloat16())


@pytest.mark.parametrize("M,N,E,K", [(1 << 25, 256, 1024, 16), (1 << 16, 1 << 17, 3, 16), (1 << 25, 1, 1, 20)])
def test_groups_of_as_many_results_as_are_taken(M, N, E, K):
    """Ragged groups, some of them empty; rows by number out of a thousand."""
    g = gen(4)
    x, w = small_codes(g, 1000, K), small_codes(g, E * N, K).view(E, N, K)
    cut = torch.randint(0, M + 1, (E - 1,), generator=g, device=DEV).sort()[0]
    if E > 8:
        cut[5:8] = cut[5].clone()
    offsets = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), M)]).int()
    rows = torch.randint(0, 1000, (M,), generator=g, device=DEV, dtype=torch.int32)
    s, ws = ones(1000, K), torch.ones((E, -(-N // 128), 1), device=DEV)
    y = new(M, N, dtype=torch.bfloat16)
    y.fill_(77)
    torch.cuda.synchronize()
    abi.moe_grouped_linear(x, abi.DT_FP8, K, s, 1, 1000, rows, offsets, E, M, w, K, N * K, ws, 1, ws.shape[1], N, K, y, abi.DT_BF16, N)
    torch.cuda.synchronize()
    at = offsets.tolist()
    step = max(1, (1 << 29) // N)
    for e in range(E):
        each = (x.float() @ w[e].float().t().contiguous()).bfloat16()      # of the thousand rows
        for i in range(at[e], at[e + 1], step):
            j = min(i + step, at[e + 1])
            assert torch.equal(y[i:j], each[rows[i:j].long()])


@pytest.mark.parametrize("E", [3, 1024])
def test_grouping_of_as_many_ids_as_are_taken(E):
    T, k = 1 << 20, 32
    g = gen(5)
    idx = torch.randint(-1, E + 1, (T, k), generator=g, device=DEV, dtype=torch.int32)
    offsets, rows, pos = (new(n, dtype=torch.int32) for n in (E + 1, T * k, T * k))
    for t in (offsets, rows, pos):
        t.fill_(-77)
    torch.cuda.synchronize()
    abi.moe_group_rows(idx, T, k, E, offsets, rows, pos)
    torch.cuda.synchronize()
    flat = idx.view(-1).long()
    ok = (flat >= 0) & (flat < E)
    where = ok.nonzero().view(-1)
    order = where[flat[where].sort(stable=True)[1]]
    want = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    want[1:] = torch.bincount(flat[where], minlength=E).cumsum(0)
    assert torch.equal(offsets.long(), want)
    n = order.numel()
    assert torch.equal(rows[:n].long(), order // k) and bool((rows[n:] == -77).all())
    place = torch.full((T * k,), -1, dtype=torch.int64, device=DEV)
    place[order] = torch.arange(n, device=DEV)
    assert torch.equal(pos.long(), place)


@pytest.mark.parametrize("T,k,H", [(1 << 20, 32, 12), (2, 3, 1 << 20), (1 << 20, 1, 3)])
def test_sums_of_as_many_rows_as_are_taken(T, k, H):
    """Weights and values that are small whole numbers: sums are exact."""
    g = gen(6)
    y = torch.randint(-2, 3, (T, H), generator=g, device=DEV).bfloat16()
    pos = torch.randint(-1, T + 1, (T, k), generator=g, device=DEV, dtype=torch.int32)
    w = torch.randint(-1, 2, (T, k), generator=g, device=DEV).float()
    out = new(T, H, dtype=torch.float32)
    torch.cuda.synchronize()
    abi.moe_combine_rows(y, abi.DT_BF16, H, T, pos, w, None, 0, T, k, H, out, abi.DT_F32, H)
    torch.cuda.synchronize()
    want = torch.zeros((T, H), device=DEV)
    for i in range(k):
        p = pos[:, i].long()
        ok = (p >= 0) & (p < T)
        want += torch.where(ok, w[:, i], 0.0)[:, None] * y[p.clamp(0, T - 1)].float()
    assert torch.equal(out, want)
