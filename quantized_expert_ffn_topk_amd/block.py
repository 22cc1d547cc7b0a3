"""FFN halves of a transformer block on the GPU, driven through the C ABI.

The blocks of a DeepSeek-V3-style model are a residual stream with two kinds of
FFN half: the first layers dense, the others a routed MoE layer, each behind an
RMS norm that takes the residual's addition.

    DenseFFN.forward:  moe_rmsnorm_quant -> moe_linear_int8 (gate and up) ->
                       moe_swiglu_quant -> moe_linear_int8 (down)
    MoEFFN.forward:    moe_rmsnorm_quant -> moe_router_topk_grouped ->
                       moe_expert_ffn

and the same two with E4M3 weights (a scale for each block of 128 x 128):

    Fp8DenseFFN.forward:  moe_rmsnorm_quant -> moe_quant_fp8 -> moe_linear_fp8 ->
                          moe_quant_fp8 (SwiGLU) -> moe_linear_fp8
    Fp8MoEFFN.forward:    moe_rmsnorm_quant -> moe_grouped_linear (the router's
                          logits) -> moe_route_select -> moe_group_rows ->
                          moe_quant_fp8 -> moe_grouped_linear -> moe_quant_fp8
                          (SwiGLU) -> moe_grouped_linear -> moe_combine_rows, on
                          top of the shared expert's two moe_linear_fp8

All take the last half's output and the residual stream and give their own
output and the new stream, so halves follow one another:

    y, res = dense.forward(attn_out, res)
    y, res = moe.forward(attn_out, res)

torch supplies device memory and streams only.
"""
from . import abi


def _dtype(t):
    import torch
    codes = {torch.float32: abi.DT_F32, torch.bfloat16: abi.DT_BF16}
    if t.dtype not in codes:
        raise ValueError("expected fp32 or bf16, got %s" % t.dtype)
    return codes[t.dtype]


def _rows(t, name, width, dtypes=None):
    """Checks a [T, width] tensor of dense rows and returns its row stride."""
    if t.dim() != 2 or t.shape[1] != width:
        raise ValueError("%s has shape %s, expected [T, %d]" % (name, tuple(t.shape), width))
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError("the values of a row of %s must be neighbours" % name)
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError("%s is %s, expected one of %s" % (name, t.dtype, dtypes))
    # a single row may report any stride
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), width)


def quantise_weight(w):
    """int8 codes [N, K] and fp32 channel scales [N] of a weight matrix: the rule
    of the activations, per output channel.  A zero channel gets scale 0; one with
    a NaN or an infinity gets scale NaN and codes 0; one below 2^-96 is multiplied
    by 2^64 first (exact), so that 127/max stays finite."""
    import torch
    w = w.float()
    amax = w.abs().amax(dim=1)
    fine = torch.isfinite(amax)
    pre = torch.ones_like(amax).masked_fill(amax < 2.0 ** -96, 2.0 ** 64)
    inv = torch.where(fine & (amax > 0), 127.0 / (amax * pre), 0.0)
    q = torch.clamp(torch.round((w * pre[:, None]) * inv[:, None]), -127, 127)
    q = torch.where(fine[:, None], q, 0.0).to(torch.int8)
    return q.contiguous(), torch.where(fine, amax / 127.0, float("nan"))


def quantise_weight_fp8(w):
    """E4M3 codes [.., N, K] (torch.float8_e4m3fn) and scales [.., ceil(N/128), ceil(K/128)]
    of weights, by the rule of the activations (moe_quant_fp8) for each block of
    128 x 128: a zero block gets scale 0, one with a NaN or an infinity scale NaN and
    codes 0."""
    import torch
    N, K = w.shape[-2:]
    nb, kb = -(-N // 128), -(-K // 128)
    by = torch.nn.functional.pad(w.float(), (0, 128 * kb - K, 0, 128 * nb - N)).unflatten(-1, (kb, 128)).unflatten(-3, (nb, 128))
    amax = by.abs().amax(dim=(-1, -3))
    fine = torch.isfinite(amax)
    pre = torch.ones_like(amax).masked_fill(amax < 2.0 ** -96, 2.0 ** 64)
    # quotients of tensors, each rounded once: with a number, torch's are a reciprocal and a product
    top = torch.full_like(amax, 448.0)
    inv = torch.where(fine & (amax > 0), top / (amax * pre), 0.0)
    at = lambda v: v[..., :, None, :, None]  # noqa: E731
    q = torch.where(at(fine), (by * at(pre)) * at(inv), 0.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    q = q.flatten(-4, -3).flatten(-2, -1)[..., :N, :K]
    return q.contiguous(), torch.where(fine, amax / top, float("nan"))


def _blocks(n):
    return -(-n // 128)


def _fp8_weights(t, w, s, shape, name):
    """Checks E4M3 weights of a shape and their scales, and returns both as they are read."""
    if w.dtype != t.float8_e4m3fn:
        raise ValueError("%s must be E4M3 codes (torch.float8_e4m3fn), not %s" % (name, w.dtype))
    if tuple(w.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(w.shape), tuple(shape)))
    want = tuple(shape[:-2]) + (_blocks(shape[-2]), _blocks(shape[-1]))
    if tuple(s.shape) != want:
        raise ValueError("the scales of %s have shape %s, expected %s" % (name, tuple(s.shape), want))
    return w.contiguous(), s.float().contiguous()


class _Norm:
    """The norm in front of a half: gamma [H] and its outputs for up to max_tokens rows."""

    def __init__(self, gamma, max_tokens, eps):
        import torch
        if gamma.dim() != 1:
            raise ValueError("gamma must be a vector")
        if gamma.device.type != "cuda":
            raise ValueError("gamma is on %s, not on a GPU" % gamma.device)
        self.torch = torch
        self.gamma = gamma.float().contiguous()
        self.H = gamma.shape[0]
        self.dev = gamma.device
        self.eps = float(eps)
        self.max_tokens = int(max_tokens)

    def _check(self, x, residual):
        t = self.torch
        ldx = _rows(x, "x", self.H, (t.float32, t.bfloat16))
        ldr = _rows(residual, "residual", self.H, (t.float32, t.bfloat16))
        T = x.shape[0]
        if residual.shape[0] != T:
            raise ValueError("x has %d rows, the residual %d" % (T, residual.shape[0]))
        if T > self.max_tokens:
            raise ValueError("%d tokens, at most %d" % (T, self.max_tokens))
        if x.device != self.dev or residual.device != self.dev:
            raise ValueError("x and residual must be on %s" % self.dev)
        return T, ldx, ldr

    def _made(self):
        """The end of a constructor.  The object's rows and weights lie where earlier
        work of torch's current stream may still be at work, and may themselves be
        on their way: it is waited for, so that forward may use any stream."""
        t = self.torch
        home = t.cuda.current_stream(self.dev)
        home.synchronize()
        self._known = {home}
        self._own = [a for a in vars(self).values() if isinstance(a, t.Tensor)]

    def _on(self, stream, x, residual):
        """The device, and torch's current stream: what is allocated inside belongs
        to the stream that writes it.  The object's tensors and the inputs are
        recorded on a stream that is not their own, so that dropping them early does
        not give their memory away under the kernels."""
        t = self.torch
        if isinstance(stream, int):
            return t.cuda.stream(t.cuda.ExternalStream(stream, device=self.dev))
        s = t.cuda.default_stream(self.dev) if stream is None else stream
        if s.device != self.dev:
            raise ValueError("the stream is of %s, not of %s" % (s.device, self.dev))
        if s not in self._known:
            for a in self._own:
                a.record_stream(s)
            self._known.add(s)
        if s != t.cuda.current_stream(self.dev):
            x.record_stream(s)
            residual.record_stream(s)
        return t.cuda.stream(s)

    def _norm(self, x, residual, rows, y, q, s, stream):
        T, ldx, ldr = rows
        h = self.torch.empty((T, self.H), dtype=residual.dtype, device=self.dev)
        abi.moe_rmsnorm_quant(x, _dtype(x), ldx, residual, _dtype(residual), ldr, self.gamma, T, self.H,
                              self.eps, h, self.H, y, self.H, q, self.H, s, stream)
        return T, h


class DenseFFN(_Norm):
    """A dense SwiGLU FFN with int8 weights: gate_up [2F, H] (the gate rows above
    the up rows) with channel scales s_gu [2F], down [H, F] with s_dn [H]."""

    def __init__(self, gamma, gate_up, s_gu, down, s_dn, max_tokens, eps=1e-6, out_dtype=None):
        super().__init__(gamma, max_tokens, eps)
        t, H = self.torch, self.H
        if gate_up.dim() != 2 or down.dim() != 2:
            raise ValueError("gate_up and down must be matrices")
        F = down.shape[1]
        if gate_up.dtype != t.int8 or down.dtype != t.int8:
            raise ValueError("weights must be int8 codes")
        if tuple(gate_up.shape) != (2 * F, H) or down.shape[0] != H:
            raise ValueError("gate_up must be [2F, H], down [H, F]")
        if tuple(s_gu.shape) != (2 * F,) or tuple(s_dn.shape) != (H,):
            raise ValueError("a scale per output channel is needed")
        self.F = F
        self.gate_up, self.down = gate_up.contiguous(), down.contiguous()
        self.s_gu, self.s_dn = s_gu.float().contiguous(), s_dn.float().contiguous()
        if any(a.device != self.dev for a in (self.gate_up, self.down, self.s_gu, self.s_dn)):
            raise ValueError("weights and gamma must be on one device")
        self.out_dtype = out_dtype or t.bfloat16
        if self.out_dtype not in (t.float32, t.bfloat16):
            raise ValueError("out_dtype must be fp32 or bf16, not %s" % self.out_dtype)
        n = self.max_tokens
        e = lambda *shape, dt: t.empty(shape, dtype=dt, device=self.dev)  # noqa: E731
        self.q, self.s = e(n, H, dt=t.int8), e(n, dt=t.float32)
        self.gu = e(n, 2 * F, dt=t.bfloat16)
        self.qh, self.sh = e(n, F, dt=t.int8), e(n, dt=t.float32)
        self._made()

    def forward(self, x, residual, stream=None):
        """(output [T, H], new residual [T, H]); enqueued on `stream` (None: the
        null stream), which the inputs must be ready on and the outputs belong
        to: whoever reads them on another stream waits for this one, and records
        them there before dropping them.  One call at a time: the intermediate
        rows are the object's own, so a call on another stream has to wait for the
        last one.  A raw handle of a stream says nothing about how long it lives:
        with one, the inputs and the object are kept until its work is done."""
        H, F = self.H, self.F
        rows = self._check(x, residual)
        with self._on(stream, x, residual):
            T, h = self._norm(x, residual, rows, None, self.q, self.s, stream)
            out = self.torch.empty((T, H), dtype=self.out_dtype, device=self.dev)
            abi.moe_linear_int8(self.q, H, self.s, T, self.gate_up, H, self.s_gu, None, 2 * F, H, self.gu,
                                abi.DT_BF16, 2 * F, stream)
            abi.moe_swiglu_quant(self.gu, abi.DT_BF16, 2 * F, T, F, None, 0, self.qh, F, self.sh, stream)
            abi.moe_linear_int8(self.qh, F, self.sh, T, self.down, F, self.s_dn, None, H, F, out,
                                _dtype(out), H, stream)
        return out, h


class MoEFFN(_Norm):
    """A routed FFN half: the norm, the choice of experts by `route` (a
    moe_route_desc whose top_k is the layer's) and the experts of `layer` (a
    layer.Layer)."""

    def __init__(self, gamma, layer, route, eps=1e-6):
        super().__init__(gamma, layer.max_tokens, eps)
        if layer.dev != self.dev:
            raise ValueError("the layer is on %s, gamma on %s" % (layer.dev, self.dev))
        if layer.desc.hidden != self.H:
            raise ValueError("the layer's hidden is %d, gamma has %d" % (layer.desc.hidden, self.H))
        if route.top_k != layer.desc.top_k or route.n_experts != layer.desc.n_experts:
            raise ValueError("the route's experts and top_k must be the layer's")
        self.layer, self.route = layer, route
        t = self.torch
        self.y = t.empty((self.max_tokens, self.H), dtype=t.bfloat16, device=self.dev)
        self.idx = t.empty((self.max_tokens, route.top_k), dtype=t.int32, device=self.dev)
        self.w = t.empty((self.max_tokens, route.top_k), dtype=t.float32, device=self.dev)
        self._made()

    def forward(self, x, residual, stream=None):
        """As DenseFFN.forward; the chosen experts and their weights are in
        idx[:T] and w[:T] afterwards."""
        odt = self.torch.bfloat16 if self.layer.desc.out_dtype == abi.DT_BF16 else self.torch.float32
        rows = self._check(x, residual)
        with self._on(stream, x, residual):
            T, h = self._norm(x, residual, rows, self.y, None, None, stream)
            out = self.torch.empty((T, self.H), dtype=odt, device=self.dev)
            abi.moe_router_topk_grouped(self.layer.ctx, self.route, self.y, T, self.layer.weights, self.idx,
                                        self.w, stream)
            abi.moe_expert_ffn(self.layer.ctx, self.y, T, self.layer.weights, self.idx, self.w, out, stream)
        return out, h


class _Fp8FFN:
    """A SwiGLU FFN of E4M3 weights between codes and rows: gate_up [2F, H] with s_gu,
    down [H, F] with s_dn, and the rows between its products for up to max_tokens rows."""

    def __init__(self, H, dev, gate_up, s_gu, down, s_dn, max_tokens):
        import torch as t
        if gate_up.dim() != 2 or down.dim() != 2:
            raise ValueError("gate_up and down must be matrices")
        self.H, F = H, down.shape[1]
        self.F = F
        self.gate_up, self.s_gu = _fp8_weights(t, gate_up, s_gu, (2 * F, H), "gate_up")
        self.down, self.s_dn = _fp8_weights(t, down, s_dn, (H, F), "down")
        if any(a.device != dev for a in (self.gate_up, self.down, self.s_gu, self.s_dn)):
            raise ValueError("weights and gamma must be on one device")
        e = lambda *shape, dt: t.empty((max_tokens,) + shape, dtype=dt, device=dev)  # noqa: E731
        self.gu = e(2 * F, dt=t.bfloat16)
        self.qh, self.sh = e(F, dt=t.float8_e4m3fn), e(_blocks(F), dt=t.float32)

    def products(self, T, q, s, out, stream):
        """out [T, H] from codes q [T, H] with scales s."""
        H, F, hb, fb = self.H, self.F, _blocks(self.H), _blocks(self.F)
        abi.moe_linear_fp8(q, H, s, hb, T, self.gate_up, H, self.s_gu, hb, None, 2 * F, H, self.gu, abi.DT_BF16, 2 * F, stream)
        abi.moe_quant_fp8(self.gu, abi.DT_BF16, 2 * F, abi.ACT_SWIGLU, T, F, None, self.qh, F, self.sh, fb, stream)
        abi.moe_linear_fp8(self.qh, F, self.sh, fb, T, self.down, F, self.s_dn, fb, None, H, F, out, _dtype(out), H, stream)


class Fp8DenseFFN(_Norm, _Fp8FFN):
    """A dense SwiGLU FFN with E4M3 weights: gate_up [2F, H] (the gate rows above the
    up rows) with scales s_gu [ceil(2F/128), ceil(H/128)], down [H, F] with s_dn
    [ceil(H/128), ceil(F/128)] (quantise_weight_fp8 makes them)."""

    def __init__(self, gamma, gate_up, s_gu, down, s_dn, max_tokens, eps=1e-6, out_dtype=None):
        _Norm.__init__(self, gamma, max_tokens, eps)
        t, H, n = self.torch, self.H, self.max_tokens
        _Fp8FFN.__init__(self, H, self.dev, gate_up, s_gu, down, s_dn, n)
        self.out_dtype = out_dtype or t.bfloat16
        if self.out_dtype not in (t.float32, t.bfloat16):
            raise ValueError("out_dtype must be fp32 or bf16, not %s" % self.out_dtype)
        e = lambda *shape, dt: t.empty(shape, dtype=dt, device=self.dev)  # noqa: E731
        self.y = e(n, H, dt=t.bfloat16)
        self.q, self.s = e(n, H, dt=t.float8_e4m3fn), e(n, _blocks(H), dt=t.float32)
        self._made()

    def forward(self, x, residual, stream=None):
        """As DenseFFN.forward."""
        H = self.H
        rows = self._check(x, residual)
        with self._on(stream, x, residual):
            T, h = self._norm(x, residual, rows, self.y, None, None, stream)
            out = self.torch.empty((T, H), dtype=self.out_dtype, device=self.dev)
            abi.moe_quant_fp8(self.y, abi.DT_BF16, H, abi.ACT_NONE, T, H, None, self.q, H, self.s, _blocks(H), stream)
            self.products(T, self.q, self.s, out, stream)
        return out, h


class Fp8MoEFFN(_Norm):
    """A routed FFN half with E4M3 experts: the norm, the router's logits from router
    [E, H] (bf16), the choice of experts by `route` (a moe_route_desc) with bias [E] or
    None, and the experts gate_up [E, 2F, H] with s_gu [E, ceil(2F/128), ceil(H/128)],
    down [E, H, F] with s_dn [E, ceil(H/128), ceil(F/128)].  `shared`: None, or (gate_up,
    s_gu, down, s_dn) of an expert that every token takes, of any F."""

    def __init__(self, gamma, router, bias, gate_up, s_gu, down, s_dn, route, max_tokens, shared=None, eps=1e-6,
                 out_dtype=None):
        super().__init__(gamma, max_tokens, eps)
        t, H = self.torch, self.H
        E, k = route.n_experts, route.top_k
        if gate_up.dim() != 3 or down.dim() != 3:
            raise ValueError("gate_up and down must be stacks of the experts' matrices")
        F = self.F = down.shape[2]
        self.gate_up, self.s_gu = _fp8_weights(t, gate_up, s_gu, (E, 2 * F, H), "gate_up")
        self.down, self.s_dn = _fp8_weights(t, down, s_dn, (E, H, F), "down")
        if tuple(router.shape) != (E, H) or router.dtype != t.bfloat16:
            raise ValueError("router must be bf16 [%d, %d]" % (E, H))
        if bias is not None and tuple(bias.shape) != (E,):
            raise ValueError("bias must have a value for each expert")
        self.router = router.contiguous()
        self.bias = None if bias is None else bias.float().contiguous()
        own = [self.gate_up, self.s_gu, self.down, self.s_dn, self.router] + ([] if bias is None else [self.bias])
        if any(a.device != self.dev for a in own):
            raise ValueError("weights and gamma must be on one device")
        self.out_dtype = out_dtype or t.bfloat16
        if self.out_dtype not in (t.float32, t.bfloat16):
            raise ValueError("out_dtype must be fp32 or bf16, not %s" % self.out_dtype)
        self.route = route
        self.shared = None
        if shared is not None:
            self.shared = _Fp8FFN(H, self.dev, *shared, max_tokens=self.max_tokens)
        n, m = self.max_tokens, self.max_tokens * k
        e = lambda *shape, dt: t.empty(shape, dtype=dt, device=self.dev)  # noqa: E731
        self.y, self.logits = e(n, H, dt=t.bfloat16), e(n, E, dt=t.float32)
        self.idx, self.w = e(n, k, dt=t.int32), e(n, k, dt=t.float32)
        # one group of all rows: its end is taken as their number
        self.whole = t.tensor([0, 2 ** 31 - 1], dtype=t.int32, device=self.dev)
        self.offsets, self.rows, self.pos = e(E + 1, dt=t.int32), e(m, dt=t.int32), e(m, dt=t.int32)
        self.q, self.s = e(n, H, dt=t.float8_e4m3fn), e(n, _blocks(H), dt=t.float32)
        self.gu, self.yr = e(m, 2 * F, dt=t.bfloat16), e(m, H, dt=t.bfloat16)
        self.qh, self.sh = e(m, F, dt=t.float8_e4m3fn), e(m, _blocks(F), dt=t.float32)
        self._made()
        if self.shared is not None:
            self._own += [a for a in vars(self.shared).values() if isinstance(a, t.Tensor)]

    def forward(self, x, residual, stream=None):
        """As DenseFFN.forward; the chosen experts and their weights are in idx[:T] and
        w[:T] afterwards."""
        H, F, E, k = self.H, self.F, self.route.n_experts, self.route.top_k
        hb, fb = _blocks(H), _blocks(F)
        rows = self._check(x, residual)
        with self._on(stream, x, residual):
            T, h = self._norm(x, residual, rows, self.y, None, None, stream)
            M = T * k
            out = self.torch.empty((T, H), dtype=self.out_dtype, device=self.dev)
            abi.moe_grouped_linear(self.y, abi.DT_BF16, H, None, 0, T, None, self.whole, 1, T, self.router, H, E * H, None, 0, 0,
                                   E, H, self.logits, abi.DT_F32, E, stream)
            abi.moe_route_select(self.route, self.logits, abi.DT_F32, E, self.bias, T, self.idx, self.w, stream)
            abi.moe_group_rows(self.idx, T, k, E, self.offsets, self.rows, self.pos, stream)
            abi.moe_quant_fp8(self.y, abi.DT_BF16, H, abi.ACT_NONE, T, H, None, self.q, H, self.s, hb, stream)
            abi.moe_grouped_linear(self.q, abi.DT_FP8, H, self.s, hb, T, self.rows, self.offsets, E, M, self.gate_up, H,
                                   2 * F * H, self.s_gu, hb, _blocks(2 * F) * hb, 2 * F, H, self.gu, abi.DT_BF16, 2 * F, stream)
            abi.moe_quant_fp8(self.gu, abi.DT_BF16, 2 * F, abi.ACT_SWIGLU, M, F, self.offsets[E:], self.qh, F, self.sh, fb, stream)
            abi.moe_grouped_linear(self.qh, abi.DT_FP8, F, self.sh, fb, M, None, self.offsets, E, M, self.down, F, H * F,
                                   self.s_dn, fb, hb * fb, H, F, self.yr, abi.DT_BF16, H, stream)
            if self.shared is not None:
                self.shared.products(T, self.q, self.s, out, stream)
            # the shared expert's rows are of out's type: a bf16 output rounds them once more (2^-8 of
            # them at most, as its own rounding), an fp32 one does not
            abi.moe_combine_rows(self.yr, abi.DT_BF16, H, M, self.pos, self.w, out if self.shared is not None else None, H, T, k, H,
                                 out, _dtype(out), H, stream)
        return out, h
