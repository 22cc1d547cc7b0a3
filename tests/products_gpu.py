"""Cases of products_cases on the GPU: inputs made on the device, the library's call, and the product in 64 bits there
with the bounds that fp8_ref derives (limit; here on device tensors, for whole results)."""
import torch

from quantized_expert_ffn_topk_amd import abi
from tests import fp8_ref as ref
from tests import products_cases as pc

DEV = "cuda"
FP8 = torch.float8_e4m3fn
DT = {"f32": abi.DT_F32, "bf16": abi.DT_BF16, "fp8": abi.DT_FP8}
TDT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}
CANARY = 77
NONE = {torch.uint8: 0x7f, torch.bfloat16: float("nan"), torch.float32: float("nan")}    # between the rows


def limit(x, w, size, out_bf16, unit_fp8):
    """fp8_ref.limit of values x [T,K], w [N,K] in 64 bits."""
    K = x.shape[1]
    x, w, want = x.abs(), w.abs(), x @ w.t().contiguous()
    P = x @ w.t().contiguous()
    lim = (32 + K / 32 + 4 * ref.blocks(K) + 19 + ref.blocks(K * size)) * 2 * ref.U * P
    if unit_fp8:
        top = torch.zeros_like(P)
        for k in range(0, K, 8):
            xe, we = x[:, k:k + 8].t().contiguous(), w[:, k:k + 8].t().contiguous()
            each = torch.outer(xe[0], we[0])
            for j in range(1, xe.shape[0]):
                each = torch.maximum(each, torch.outer(xe[j], we[j]))
            top += each
        lim += 8 * 2.0 ** -13 * top
    if out_bf16:
        lim = lim * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    return lim + 1e-37


def spread(s, n):
    return s.double().repeat_interleave(ref.BLOCK, dim=-1)[..., :n]


def rows_apart(n, row, dtype, ld, shift=0):
    """[n, row] on the device, `ld` elements apart, NaN between the rows and in front of the first where that is no
    great memory."""
    count = (n - 1) * ld + row + shift
    flat = torch.empty(count, dtype=dtype, device=DEV) if count > 1 << 28 else torch.full((count,), NONE[dtype], dtype=dtype, device=DEV)
    return flat.as_strided((n, row), (ld, 1), shift)


class Product:
    """Inputs of a case.  x and w are what is passed, xv and wv(e) the values that they stand for."""

    def __init__(self, c, seed=1):
        self.c, self.grouped = c, "sizes" in c
        self.kernel = pc.kernel(c)
        assert pc.name_of(self.kernel) == c["name"]
        g = self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.N, self.K, self.out = c["N"], c["K"], c["out"]
        self.xd = c.get("xd", "fp8")
        self.E = len(c["sizes"]) if self.grouped else 1
        self.sizes = list(c["sizes"]) if self.grouped else [c["T"]]
        self.M, self.R = sum(self.sizes), pc.rows_of_x(c)
        self.kb, self.nb = ref.blocks(self.K), ref.blocks(self.N)
        shift = c.get("shift", 0)
        stride = {n: pc.ld(c, n) for n in ("ldx", "ldw", "lds", "ldws", "ldo", "w_stride", "ws_stride")}
        self.stride = stride
        self.offsets = torch.tensor([0] + self.sizes, device=DEV).cumsum(0).int()
        self.rows = None
        if self.grouped and c["gather"]:
            self.rows = torch.randint(0, self.R, (self.M,), generator=g, device=DEV, dtype=torch.int32)
        self.x = rows_apart(self.R, self.K, TDT[self.xd], stride["ldx"], shift)
        self.fill(self.x)
        self.w = self.stack(self.K, self.N, TDT[self.xd], stride["ldw"], stride["w_stride"], shift)
        for e in range(self.E):
            self.fill(self.w[e], 0.1)
        self.s = self.ws = None
        if self.xd == "fp8":
            self.s = rows_apart(self.R, self.kb, torch.float32, stride["lds"])
            self.ws = self.stack(self.kb, self.nb, torch.float32, stride["ldws"], stride["ws_stride"])
            self.scales(self.s, -9.0)
            for e in range(self.E):
                self.scales(self.ws[e], -14.0)
        self.bias = None
        if not self.grouped and shift:
            self.bias = torch.randn(self.N, generator=g, device=DEV)
        self.flat, self.y = None, None

    def stack(self, row, n, dtype, ld, stride, shift=0):
        flat = rows_apart(1, (self.E - 1) * stride + (n - 1) * ld + row, dtype, 1, shift)
        return flat.as_strided((self.E, n, row), (stride, ld, 1), shift)

    def fill(self, to, scale=1.0):
        step = max(1, (1 << 26) // self.K)
        for i in range(0, to.shape[0], step):
            v = torch.randn((min(step, to.shape[0] - i), self.K), generator=self.g, device=DEV)
            to[i:i + step] = (v * 150).clamp_(-448, 448).to(FP8).view(torch.uint8) if self.xd == "fp8" else v.mul_(scale).bfloat16()

    def scales(self, to, low):
        to.copy_(2.0 ** (low + 3 * torch.rand(to.shape, generator=self.g, device=DEV)))

    def fresh(self):
        """Rows of out with a canary everywhere."""
        ld, n = self.stride["ldo"], (self.M - 1) * self.stride["ldo"] + self.N
        if n > 1 << 28:
            self.flat = torch.empty(n, dtype=TDT[self.out], device=DEV)
        else:
            self.flat = torch.full((n + 64,), CANARY, dtype=TDT[self.out], device=DEV)
        self.y = self.flat.as_strided((self.M, self.N), (ld, 1))
        self.y.fill_(CANARY)

    def call(self, y=None, stream=None, offsets=None, rows=None):
        st, y = self.stride, self.y if y is None else y
        if self.grouped:
            abi.moe_grouped_linear(self.x, DT[self.xd], st["ldx"], self.s, st["lds"], self.R, self.rows if rows is None else rows,
                                   self.offsets if offsets is None else offsets, self.E, self.M, self.w, st["ldw"],
                                   st["w_stride"], self.ws, st["ldws"], st["ws_stride"], self.N, self.K, y, DT[self.out], st["ldo"],
                                   stream)
        else:
            abi.moe_linear_fp8(self.x, st["ldx"], self.s, st["lds"], self.M, self.w, st["ldw"], self.ws, st["ldws"], self.bias,
                               self.N, self.K, y, DT[self.out], st["ldo"], stream)

    def run(self, **more):
        self.fresh()
        torch.cuda.synchronize()
        self.call(**more)
        torch.cuda.synchronize()
        return self.y

    def value(self, codes, s):
        return codes.view(FP8).double() * s if self.xd == "fp8" else codes.double()

    def xv(self, at):
        return self.value(self.x[at].contiguous(), None if self.s is None else spread(self.s[at], self.K))

    def wv(self, e):
        s = None if self.ws is None else spread(self.ws[e].repeat_interleave(ref.BLOCK, dim=0)[:self.N], self.K)
        return self.value(self.w[e].contiguous(), s)

    def check(self, y):
        """Every value of y against the product in 64 bits; what lies between and behind the rows is untouched."""
        if self.flat.numel() <= 1 << 28:
            rest = self.flat.clone()
            rest.as_strided(self.y.shape, self.y.stride()).fill_(CANARY)
            assert (rest == CANARY).all()
        o = [0]
        for n in self.sizes:
            o.append(o[-1] + n)
        for e in range(self.E):
            if o[e] == o[e + 1]:
                continue
            at = slice(o[e], o[e + 1]) if self.rows is None else self.rows[o[e]:o[e + 1]].long()
            x, w = self.xv(at), self.wv(e)
            want = x @ w.t().contiguous()
            lim = limit(x, w, 2 if self.xd == "bf16" else 1, self.out == "bf16", self.kernel.unit == "f8")
            if self.bias is not None:
                want = want + self.bias.double()
                lim = lim + (2 * ref.U + (2.0 ** -8 if self.out == "bf16" else 0)) * self.bias.double().abs()
            off = (y[o[e]:o[e + 1]].double() - want).abs()
            assert bool((off <= lim).all()), (e, float((off - lim).max()))
