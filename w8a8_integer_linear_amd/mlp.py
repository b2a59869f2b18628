"""A feed-forward block in quantized training: two INT8 W8A8 projections with an
activation, mostly gated, between them, as a sequence of C-ABI calls.

Both weights are INT8 codes with a float magnitude per row and no float master copy
(mini_trainer guide), in the rotated basis of OneTrainer PR #1681, and are updated
by the layer's own stochastic requantization.

Step order of one training step:
  forward   qlin_quantize_rows(x, rotate)               -> qx, sx            (saved)
            qlin_fwd_gated(qx, W1) or qlin_fwd_act      -> h, ck, ck_s       (ck saved)
            qlin_quantize_rows(h, rotate)               -> qh, sh            (saved)
            qlin_fwd_act(qh, W2, residual)              -> y
  backward  qlin_quantize_grad(dy, sw2, sh)             -> its codes, db2
            qlin_product_ws(DX), qlin_product_ws(DW)    -> dh, dw2
            qlin_act_bwd(dh, ck, sw1, sx)               -> dz, s1, s2, db1
            qlin_quantize_grad_scaled(dz, s1, s2)       -> its codes
            qlin_product_ws(DX), qlin_product_ws(DW)    -> dx, dw1
  update    qlin_sgd_requant or qlin_adamw_requant, both weights

Kept between forward and backward are three arrays of codes, one byte per element of
x, h and the sums before the activation; the sums themselves, and h, are not.
"""
import torch

from . import _native as nat
from .layer import LinearW8A8Training


class MLPW8A8Training:
    def __init__(self, w1, w2, b1=None, b2=None, act="gelu", gated=False, had_block=128,
                 dtype=torch.bfloat16):
        """w1: [F, K], with a gate [2 F, K] (the gate's rows first); w2: [N, F]; float GPU
        tensors in the original basis.  b1, b2: biases or None.  act: a name of
        ACTIVATIONS.  dtype: of h and of its gradient dz between the products (float32
        or bfloat16).  A w1 of more than MAX_ROW rows serves only: its gradient's rows
        are longer than quantization takes."""
        nat._act_code(act)
        rows, self.K = w1.shape
        self.N, self.F = w2.shape
        if rows != (2 * self.F if gated else self.F):
            raise ValueError(f"w1 {tuple(w1.shape)} and w2 {tuple(w2.shape)} do not fit"
                             + (" a gated block" if gated else ""))
        self.act, self.gated, self.had, self.dtype = act, bool(gated), int(had_block), dtype
        self.fc1 = LinearW8A8Training(w1, b1, had_block=had_block)
        self.fc2 = LinearW8A8Training(w2, b2, had_block=had_block)
        self.saved = None               # what the last forward left for its backward
        self._ws = {}                   # products' workspaces by stream

    def _workspace(self, M):
        """The current stream's workspace for the block's products at M tokens, grown
        (zero-filled) as needed: calls that share one must not overlap in time, and
        streams do.  In a graph's capture None: each call makes one of the graph's own,
        which no later growth frees under its replays."""
        if torch.cuda.is_current_stream_capturing():
            return None
        rows1 = self.fc1.N
        need = max(nat.qlin_product_ws_bytes(op, M, n, k)
                   for op in (nat.QLIN_OP_FWD, nat.QLIN_OP_DX, nat.QLIN_OP_DW)
                   for n, k in ((rows1, self.K), (self.N, self.F)))
        stream = nat._stream(None)
        ws = self._ws.get(stream)
        if ws is None or ws.numel() < need:
            ws = self._ws[stream] = torch.zeros(need, dtype=torch.uint8, device=self.fc1.qw.device)
        return ws

    def forward(self, x, residual=None, save=True):
        """x: [M, K], fp32 or bf16; residual: [M, N], fp32 or bf16, or None.  Returns y
        [M, N], the residual's type or x's.  What backward needs of this pass is left in
        self.saved, or self.saved is left alone (save=False: evaluation, serving)."""
        if nat._elsewhere(x, None):         # another device than the current one
            with nat._there(x, None):
                return self.forward(x, residual, save)
        M = x.shape[0]
        fc1, fc2, ws = self.fc1, self.fc2, self._workspace(M)
        qx, sx = nat.qlin_quantize_rows(x, had_block=self.had)
        first = nat.qlin_fwd_gated if self.gated else nat.qlin_fwd_act
        h, ck, ck_s = first(qx, sx, fc1.qw, fc1.sw, bias=fc1.bias, act=self.act, dtype=self.dtype,
                            save=save, workspace=ws)
        qh, sh = nat.qlin_quantize_rows(h, had_block=self.had)
        y, _, _ = nat.qlin_fwd_act(qh, sh, fc2.qw, fc2.sw, bias=fc2.bias, residual=residual,
                                   dtype=x.dtype if residual is None else residual.dtype, workspace=ws)
        if save:
            self.saved = dict(qx=qx, sx=sx, ck=ck, ck_s=ck_s, qh=qh, sh=sh)
        return y

    def backward(self, dy, saved=None):
        """dy: [M, N], fp32 or bf16.  saved: what the forward pass in question left in
        self.saved, by default the last one's.  Returns dx [M, K] fp32 in the original
        basis (the residual's gradient is dy); keeps both layers' dw and db for the
        update."""
        c = self.saved if saved is None else saved
        if c is None:
            raise RuntimeError("backward needs a forward pass before it (save=True)")
        if self.fc1.N > nat.MAX_ROW:        # (before the first gradient is overwritten)
            raise ValueError(f"backward: w1 has {self.fc1.N} rows, at most {nat.MAX_ROW} are trained")
        if nat._elsewhere(dy, None):
            with nat._there(dy, None):
                return self.backward(dy, c)
        fc1, fc2 = self.fc1, self.fc2
        M, ws = c["qx"].shape[0], self._workspace(c["qx"].shape[0])
        q1, s1, q2, s2, _ = nat.qlin_quantize_grad(dy, fc2.sw, c["sh"], col_sum=fc2.db)
        dh = nat.qlin_product_ws(nat.QLIN_OP_DX, q1, s1, fc2.qw, M, self.N, self.F, had_block=self.had,
                                 workspace=ws)
        nat.qlin_product_ws(nat.QLIN_OP_DW, q2, s2, c["qh"], M, self.N, self.F, out=fc2.dw, workspace=ws)
        dz, s1, s2, _ = nat.qlin_act_bwd(dh, c["ck"], c["ck_s"], self.act, gated=self.gated, sw=fc1.sw,
                                         sx=c["sx"], dtype=self.dtype, db=fc1.db)
        q1, q2 = nat.qlin_quantize_grad_scaled(dz, fc1.sw, c["sx"], s1, s2)
        dx = nat.qlin_product_ws(nat.QLIN_OP_DX, q1, s1, fc1.qw, M, fc1.N, self.K, had_block=self.had,
                                 workspace=ws)
        nat.qlin_product_ws(nat.QLIN_OP_DW, q2, s2, c["qx"], M, fc1.N, self.K, out=fc1.dw, workspace=ws)
        return dx

    def sgd_step(self, lr, seed, step):
        """SGD with stochastic requantization of both weights; the second's rounding
        takes the next seed."""
        self.fc1.sgd_step(lr, seed, step)
        self.fc2.sgd_step(lr, seed + 1, step)

    def adamw_step(self, lr, seed, step, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0):
        """AdamW with stochastic requantization of both weights (step >= 1)."""
        self.fc1.adamw_step(lr, seed, step, betas, eps, weight_decay)
        self.fc2.adamw_step(lr, seed + 1, step, betas, eps, weight_decay)
