"""GPU tests of every kernel that the products of E4M3 and bf16 rows can take, on the cases of products_cases: long
rows, rows far apart, NaN codes and scales, lists that are none, captures and other streams, in tiles and groups'
tiles as well as in streams."""
import pytest

from tests import products_cases as pc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.products_gpu import CANARY, DEV, Product  # noqa: E402


@pytest.mark.parametrize("case", pc.DENSE, ids=pc.label)
def test_dense_kernels(case):
    p = Product(case)
    p.check(p.run())


@pytest.mark.parametrize("case", pc.GROUPED, ids=pc.label)
def test_grouped_kernels(case):
    p = Product(case)
    p.check(p.run())


@pytest.mark.parametrize("case", pc.FAR, ids=pc.label)
def test_rows_far_apart(case):
    p = Product(case)
    p.check(p.run())


@pytest.mark.parametrize("name", sorted(pc.TILES))
def test_kernels_of_the_other_tests(name):
    p = Product(pc.TILES[name])
    p.check(p.run())


def none_of(p):
    return float("nan") if p.xd == "bf16" else 0x7f


@pytest.mark.parametrize("name", sorted(pc.TILES))
def test_codes_and_scales_that_are_no_numbers(name):
    """A NaN code, or a NaN scale, reaches its own rows or channels of its own expert and no other; rows of x that
    belong to no group reach nothing."""
    p = Product(pc.TILES[name])
    clean = p.run().clone()
    bad = torch.zeros((p.M, p.N), dtype=torch.bool, device=DEV)
    source = torch.arange(p.M, device=DEV) if p.rows is None else p.rows.long()
    first = [0]
    for n in p.sizes:
        first.append(first[-1] + n)
    of = torch.repeat_interleave(torch.arange(p.E, device=DEV), torch.tensor(p.sizes, device=DEV))

    def spoil_row(r):
        bad[source == r] = True

    def spoil_weights(e, channels):
        bad[(of == e)[:, None] & channels[None]] = True

    n = torch.arange(p.N, device=DEV)
    a, b, c = (int(source[i]) for i in (0, p.M // 2, p.M - 1))
    p.x[a, p.K - 1] = none_of(p)
    spoil_row(a)
    p.x[b, 130] = none_of(p)
    spoil_row(b)
    e = max(range(p.E), key=lambda i: p.sizes[i])
    p.w[e, 5, 3] = none_of(p)
    spoil_weights(e, n == 5)
    last = max(i for i in range(p.E) if p.sizes[i])
    p.w[last, p.N - 1, p.K - 1] = none_of(p)
    spoil_weights(last, n == p.N - 1)
    if p.xd == "fp8":
        p.s[c, 2] = float("nan")
        spoil_row(c)
        p.ws[e, 1, p.kb - 1] = float("nan")
        spoil_weights(e, n // 128 == 1)
    unused = torch.ones(p.R, dtype=torch.bool, device=DEV)
    unused[source] = False
    p.x[unused] = none_of(p)
    y = p.run()
    assert torch.equal(y.isnan(), bad)
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("name", sorted(n for n in pc.TILES if "sizes" in pc.TILES[n]))
def test_lists_that_are_none_touch_nothing_outside(name):
    """Offsets and rows of any content: nothing outside of out's rows is written, and as many rows as there were are
    there for the next call."""
    p = Product(pc.TILES[name])
    g = torch.Generator(device=DEV).manual_seed(2)
    for _ in range(3):
        wild = torch.tensor([-(1 << 31), -1, 0, 5, p.M // 2, p.M, p.M + 1, (1 << 31) - 1], device=DEV)
        offsets = wild[torch.randint(0, 8, (p.E + 1,), generator=g, device=DEV)].int()
        strange = torch.tensor([-(1 << 31), -1, 0, p.R, (1 << 31) - 1], device=DEV)
        rows = strange[torch.randint(0, 5, (p.M,), generator=g, device=DEV)].int() if p.rows is not None else None
        p.run(offsets=offsets, rows=rows)
        rest = p.flat.clone()
        rest.as_strided(p.y.shape, p.y.stride()).fill_(CANARY)
        assert (rest == CANARY).all()
    p.check(p.run())


@pytest.mark.parametrize("name", sorted(pc.TILES))
def test_on_a_side_stream_and_captured(name):
    p = Product(pc.TILES[name])
    want = p.run().clone()
    side = torch.cuda.Stream()
    assert torch.equal(p.run(stream=side), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.call(stream=torch.cuda.current_stream())
    for _ in range(3):
        p.y.fill_(CANARY)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.y, want)
        other = torch.empty_like(p.flat)                 # eager work between the replays
        p.call(y=other)
        torch.cuda.synchronize()
        assert torch.equal(other.as_strided(p.y.shape, p.y.stride()), want)
    if p.grouped:                                        # a replay goes by what the lists hold then
        p.sizes = p.sizes[::-1]
        p.offsets.copy_(torch.tensor([0] + p.sizes, device=DEV).cumsum(0).int())
        p.y.fill_(CANARY)
        graph.replay()
        torch.cuda.synchronize()
        p.check(p.y)
