"""FFN halves of a transformer block on the GPU, driven through the C ABI.

The blocks of a DeepSeek-V3-style model are a residual stream with two kinds of
FFN half: the first layers dense, the others a routed MoE layer, each behind an
RMS norm that takes the residual's addition.

    DenseFFN.forward:  moe_rmsnorm_quant -> moe_linear_int8 (gate and up) ->
                       moe_swiglu_quant -> moe_linear_int8 (down)
    MoEFFN.forward:    moe_rmsnorm_quant -> moe_router_topk_grouped ->
                       moe_expert_ffn

Both take the last half's output and the residual stream and give their own
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
