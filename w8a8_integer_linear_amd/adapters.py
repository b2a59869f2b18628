"""A frozen INT8 projection behind an RMS norm, with low-rank adapters that many
requests share: serving and training as a sequence of C-ABI calls.

A model block normalizes its residual stream and projects it.  Here the weight
stays as INT8 codes (the guide's INT8 direction with a float magnitude per
output row, in the rotated basis of OneTrainer PR #1681), and what is trained
is small and float: each adapter's two matrices and the norm's gamma.  A batch
mixes requests, each token naming its adapter (or none).

Step order:
  forward   qlin_rmsnorm_quant(x, residual)           -> h, qx, sx, rstd  (saved)
            qlin_adapter_fwd(qx, sx, qw, sw, a, b, ids) -> y, u           (u saved)
  backward  qlin_quantize_rows(dy, prescale=sw)       -> qg1, sg1
            qlin_adapter_bwd(dy, ..., order, start)   -> dx, da, db
            qlin_rmsnorm_bwd(dx, h, rstd, dres)       -> dh, dgamma
  update    qlin_adamw_tensors(a, b, gamma)           one launch

The adapters read the projection's saved codes, so a pass holds its input
once, in one byte per element.  Outputs and what a forward pass saves are
ordinary tensors; the layer itself keeps its parameters, their gradients and
moments, and one workspace per stream, however many token counts it has seen.
Forward passes may run on several streams at once; the gradients are one set, so
backward passes may not.
"""
import torch

from . import _native as nat


def pack_adapters(adapters, had_block=0, dtype=torch.float32):
    """The stacked form that qlin_adapter_fwd takes, from a list of (A [r, K],
    B [N, r], alpha) in the original basis: ranks filled up with zeros to one
    multiple of 8, A's rows rotated like the weight's, scale = alpha / r.
    Returns (a [L, R, K], b [L, N, R], scale [L])."""
    ranks = [A.shape[0] for A, _, _ in adapters]
    if not ranks or min(ranks) < 1 or max(ranks) > nat.MAX_RANK:
        raise ValueError(f"adapters need ranks of 1 to {nat.MAX_RANK}, got {ranks}")
    R = -(-max(ranks) // 8) * 8
    K, N, dev = adapters[0][0].shape[1], adapters[0][1].shape[0], adapters[0][0].device
    a = torch.zeros((len(adapters), R, K), dtype=torch.float32, device=dev)
    b = torch.zeros((len(adapters), N, R), dtype=torch.float32, device=dev)
    for l, (A, B, _) in enumerate(adapters):
        if A.shape != (ranks[l], K) or B.shape != (N, ranks[l]):
            raise ValueError(f"adapter {l}: A {tuple(A.shape)} and B {tuple(B.shape)} do not fit")
        a[l, :ranks[l]] = A
        b[l, :, :ranks[l]] = B
    if had_block:
        flat = a.view(-1, K)
        nat.qlin_hadamard(flat, had_block, y=flat)
    scale = torch.tensor([alpha / r for (_, _, alpha), r in zip(adapters, ranks)],
                         dtype=torch.float32, device=dev)
    return a.to(dtype), b.to(dtype), scale


class AdaptedLinearW8A8:
    def __init__(self, weight, gamma, adapters, bias=None, had_block=128, eps=1e-6,
                 dtype=torch.float32, state_bits=32):
        """weight: [N, K] float GPU tensor in the original basis (quantized here and
        frozen); gamma: [K]; adapters: a list of (A [r, K], B [N, r], alpha);
        dtype: of the adapters' matrices (float32 or bfloat16); state_bits: of
        their optimizer moments (32 or 8)."""
        if state_bits not in (8, 32):
            raise ValueError("state_bits is 8 or 32")
        self.N, self.K = weight.shape
        self.had, self.eps = int(had_block), float(eps)
        self.qw, self.sw = nat.qlin_quantize_rows(weight.to(torch.float32).contiguous(),
                                                  had_block=self.had)
        self.bias = None if bias is None else bias.to(torch.float32).contiguous().clone()
        self.gamma = gamma.to(torch.float32).contiguous().clone()
        self.ranks = [A.shape[0] for A, _, _ in adapters]
        self.a, self.b, self.scale = pack_adapters(adapters, self.had, dtype)
        self.L, self.R = self.a.shape[:2]
        self.da = torch.zeros(self.a.shape, dtype=torch.float32, device=self.a.device)
        self.db = torch.zeros(self.b.shape, dtype=torch.float32, device=self.a.device)
        self.dgamma = torch.zeros_like(self.gamma)
        self.state_bits = state_bits
        self._plan = None
        self.saved = None               # what the last forward left for its backward
        self._buffers = {}              # the same, by its token count and type
        self._ws = {}                   # workspaces by stream

    def _workspace(self, need):
        """The current stream's workspace, for all token counts and both directions,
        grown to need bytes (zero-filled) and never smaller: calls that share one must
        not overlap in time, and streams do.  In a graph's capture None: the call makes
        one of the graph's own, which no later growth frees under its replays."""
        if torch.cuda.is_current_stream_capturing():
            return None
        stream = nat._stream(None)
        ws = self._ws.get(stream)
        if ws is None or ws.numel() < need:
            ws = self._ws[stream] = torch.zeros(need, dtype=torch.uint8, device=self.a.device)
        return ws

    def forward(self, x, ids, residual=None, save=True):
        """x, residual: [M, K] (fp32 or bf16); ids: [M] int32, the adapter of each
        token, -1 for none.  Returns (y [M, N] fp32, h): the projection with the
        adapters, and the residual stream x + residual (x itself without one).
        y and h are the caller's.  What backward needs of this pass is left in
        self.saved, or self.saved is left alone (save=False: serving); h and ids are
        part of it and stay as they are until then."""
        M = x.shape[0]
        if save:    # (the last pass's memory may serve this one)
            self.saved, self._buffers = None, {}
        qx, sx, h, rstd, _ = nat.qlin_rmsnorm_quant(x, self.gamma, self.eps, residual=residual,
                                                    had_block=self.had)
        need = nat.qlin_adapter_fwd_ws_bytes(M, self.N, self.K, self.L, self.R)
        y, u = nat.qlin_adapter_fwd(qx, sx, self.qw, self.sw, self.a, self.b, self.scale, ids,
                                    bias=self.bias, workspace=self._workspace(need))
        if save:
            self.saved = dict(h=h, rstd=rstd, qx=qx, sx=sx, u=u, ids=ids)
            self._buffers = {(M, x.dtype): self.saved}
        return y, h

    def backward(self, dy, dres=None, saved=None):
        """dy: [M, N] (fp32 or bf16); dres: [M, K] of the stream's type, the gradient
        that reaches h past the projection.  saved: what the forward pass in question
        left in self.saved, by default the last one's (with other forward passes in
        between, keep it and hand it over).  Returns dh, the gradient of x and of the
        residual; keeps da, db and dgamma for the update."""
        c = self.saved if saved is None else saved
        if c is None:
            raise RuntimeError("backward needs a forward pass before it (save=True)")
        M = c["h"].shape[0]
        # (The gradient's codes stay beside the rest.)
        c["qg"], c["sg"] = nat.qlin_quantize_rows(dy, prescale=self.sw)
        order, start = nat.qlin_adapter_group(c["ids"], self.L)
        need = nat.qlin_adapter_bwd_ws_bytes(M, self.N, self.K, self.L, self.R)
        dx, _, _ = nat.qlin_adapter_bwd(
            dy, c["qg"], c["sg"], self.qw, c["qx"], c["sx"], c["u"], self.a, self.b, self.scale,
            c["ids"], order, start, had_block=self.had, da=self.da, db=self.db,
            workspace=self._workspace(need))
        dh, _ = nat.qlin_rmsnorm_bwd(dx, c["h"], c["rstd"], self.gamma, dres=dres,
                                     dgamma=self.dgamma)
        return dh

    def adamw_step(self, lr, seed, step, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0):
        """One AdamW step over the adapters and gamma (step >= 1).  The moments are
        allocated, zeroed, on the first call.  weight_decay is of the adapters (gamma
        has none); another value than the last step's makes a new plan."""
        if self._plan is None:
            self._trained = [self._with_moments(p, g) for p, g in (
                (self.a, self.da), (self.b, self.db), (self.gamma, self.dgamma))]
        if self._plan is None or weight_decay != self._decay:
            for t, decay in zip(self._trained, (weight_decay, weight_decay, 0.0)):
                t["weight_decay"] = decay
            self._plan, self._decay = nat.qlin_adamw_tensors_plan(self._trained), weight_decay
        nat.qlin_adamw_tensors(self._plan, lr, betas[0], betas[1], eps, seed, step)

    def _with_moments(self, p, g):
        t = dict(p=p, g=g)
        if self.state_bits == 32:
            t["m"], t["v"] = (torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                              for _ in range(2))
        else:
            for k in ("m", "v"):
                t[k] = torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(
                    torch.float8_e4m3fn)
                t[k + "_scale"] = torch.zeros(-(-p.numel() // 256), dtype=torch.float32,
                                              device=p.device)
        return t

    def adapter(self, l):
        """Adapter l's (A [r, K], B [N, r]) in the original basis, fp32."""
        r = self.ranks[l]
        A = self.a[l, :r].to(torch.float32).contiguous()
        if self.had:        # the normalized rotation is its own inverse
            A = nat.qlin_hadamard(A, self.had)
        return A, self.b[l, :, :r].to(torch.float32).contiguous()
