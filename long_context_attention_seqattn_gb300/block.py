"""One attention layer with its projections, trained chunk by chunk.

``AttentionBlock`` strings the library's calls together as a trainer of one
layer would: y = x + W_o attention(rotary(norm(x W_qkv))).  The forward runs
the chunks first to last; the backward visits them last to first (SeCO's relay
order), so the cache gradients of a chunk's rows are final right after its
own attention backward, and the rest of the chunk's graph (head norm and
rotation, projections) follows at once.  The weight gradients are summed in
float32 over the chunks, and ``step`` applies AdamW to the float32 master
weights and rewrites the bf16 ones the products read.

Host logic only: every step is a kernel of the library.
"""

import torch

from . import binding


class AttentionBlock:
    """Weights (bf16, with float32 masters), gradients and buffers of one
    layer for sequences [batch, seq_len, d_model] in bf16.

    ``plan``: rotary plan of ``binding.rope_plan`` or None; ``positions``:
    int64 [axes, batch, seq_len] on the device, or None (row r is at position
    r).  ``qk_norm``: RMS norm of query and key heads; ``bias``: a bias of the
    fused projection; ``state_bits``: of the optimizer's moments."""

    def __init__(self, batch, seq_len, d_model, num_q_heads, num_kv_heads, head_dim, chunk, plan=None,
                 positions=None, qk_norm=True, bias=False, eps=1e-6, state_bits=32, weight_decay=0.0,
                 device="cuda"):
        self.heads = (num_q_heads, num_kv_heads, num_kv_heads)
        self.head_dim, self.chunk, self.plan, self.eps = head_dim, chunk, plan, eps
        self.shape = (batch, seq_len, d_model)
        width, inner = sum(self.heads) * head_dim, num_q_heads * head_dim
        bf16 = dict(dtype=torch.bfloat16, device=device)
        self.weights = {"w_qkv": torch.zeros((d_model, width), **bf16), "w_o": torch.zeros((inner, d_model), **bf16)}
        if bias:
            self.weights["b_qkv"] = torch.zeros(width, **bf16)
        if qk_norm:
            self.weights["gamma_q"] = torch.ones(head_dim, **bf16)
            self.weights["gamma_k"] = torch.ones(head_dim, **bf16)
        self.masters = {n: w.float() for n, w in self.weights.items()}
        self.grads = {n: torch.zeros_like(w) for n, w in self.masters.items()}
        names = list(self.weights)
        self.optimizer = binding.AdamW([self.masters[n] for n in names], [self.grads[n] for n in names],
                                       lowp=[self.weights[n] for n in names], state_bits=state_bits,
                                       weight_decay=[weight_decay if n.startswith("w_") else 0.0 for n in names])
        self.qkv = torch.empty((batch, seq_len, sum(self.heads), head_dim), **bf16)
        self.k = torch.zeros((batch, seq_len, num_kv_heads, head_dim), **bf16)
        self.v = torch.zeros_like(self.k)
        self.q = torch.empty((batch, seq_len, num_q_heads, head_dim), **bf16)
        self.bufs = binding.LayerBuffers(self.q, self.k, chunk)
        self.norm_ws = torch.empty(binding.qk_norm_rope_bwd_workspace_size(head_dim), dtype=torch.uint8,
                                   device=device)
        if positions is not None and tuple(positions.shape[1:]) != (batch, seq_len):
            raise ValueError(f"positions has shape {tuple(positions.shape)}, expected [axes, {batch}, {seq_len}]")
        # a chunk's positions as one contiguous tensor, made once
        self.positions = [None if positions is None else positions[:, :, s:e].contiguous()
                          for s, e in self._chunks()]

    def _chunks(self):
        T = self.shape[1]
        return [(s, min(s + self.chunk, T)) for s in range(0, T, self.chunk)]

    def load(self, **weights):
        """Set weights by name (float32 or bf16 tensors): masters and bf16 copies."""
        for name, w in weights.items():
            self.masters[name].copy_(w)
            self.weights[name].copy_(w)

    def zero_grad(self):
        for g in self.grads.values():
            g.zero_()

    def forward(self, x):
        """y [batch, seq_len, d_model] from x (bf16); keeps what the backward reads, x among it."""
        if tuple(x.shape) != self.shape:
            raise ValueError(f"x has shape {tuple(x.shape)}, expected {self.shape}")
        w = self.weights
        y = torch.empty_like(x)
        for i, (s, e) in enumerate(self._chunks()):
            x_c = binding._rows(x, s, e)
            qkv, q, o, out = (self._chunk_buffer(t, s, e) for t in (self.qkv, self.q, self.bufs.o, y))
            binding.linear_fwd(x_c, w["w_qkv"], qkv.flatten(2), bias=w.get("b_qkv"))
            q_in, k_in, v_in = qkv.split(self.heads, 2)
            binding.qk_norm_rope_fwd(q_in, k_in, v_in, q, self.k, self.v, s, gamma_q=w.get("gamma_q"),
                                     gamma_k=w.get("gamma_k"), eps=self.eps, plan=self.plan,
                                     positions=self.positions[i])
            binding.chunk_fwd(q, self.k, self.v, o, self.bufs.lse_chunks[i], s)
            binding.linear_fwd(o.flatten(2), w["w_o"], out, residual=x_c)
            for part, whole in ((qkv, self.qkv), (q, self.q), (o, self.bufs.o), (out, y)):
                self._keep(part, whole, s, e)
        self.x = x
        return y

    def backward(self, dy):
        """dx from dy (bf16), after ``forward``; adds every weight's gradient to ``grads``."""
        if tuple(dy.shape) != self.shape:
            raise ValueError(f"dy has shape {tuple(dy.shape)}, expected {self.shape}")
        w, g, b = self.weights, self.grads, self.bufs
        dx = torch.empty_like(dy)
        binding.reset_accum(b.dk, b.dv, self.heads[0])
        for i, (s, e) in reversed(list(enumerate(self._chunks()))):
            x_c, dy_c = binding._rows(self.x, s, e), binding._rows(dy, s, e)
            qkv, q, o = (binding._rows(t, s, e) for t in (self.qkv, self.q, b.o))
            d_o, d_qkv = torch.empty_like(o), torch.empty_like(qkv)
            dq, dx_c = self._chunk_buffer(b.dq, s, e), self._chunk_buffer(dx, s, e)
            binding.linear_dgrad(dy_c, w["w_o"], d_o.flatten(2))
            binding.linear_wgrad(o.flatten(2), dy_c, g["w_o"])
            binding.chunk_bwd(q, self.k, self.v, o, b.lse_chunks[i], d_o, dq, b.dk, b.dv, s, workspace=b.workspace)
            # every later chunk has run: the rows of dk and dv are final
            q_in, k_in, _ = qkv.split(self.heads, 2)
            dq_in, dk_in, dv_in = d_qkv.split(self.heads, 2)
            binding.qk_norm_rope_bwd(q_in, k_in, dq, b.dk, b.dv, dq_in, dk_in, dv_in, s, gamma_q=w.get("gamma_q"),
                                     gamma_k=w.get("gamma_k"), dgamma_q=g.get("gamma_q"),
                                     dgamma_k=g.get("gamma_k"), eps=self.eps, plan=self.plan,
                                     positions=self.positions[i], workspace=self.norm_ws)
            binding.linear_wgrad(x_c, d_qkv.flatten(2), g["w_qkv"], dbias=g.get("b_qkv"))
            binding.linear_dgrad(d_qkv.flatten(2), w["w_qkv"], dx_c, residual=dy_c)
            self._keep(dq, b.dq, s, e)
            self._keep(dx_c, dx, s, e)
        return dx

    def step(self, lr, step, **kw):
        """One AdamW step on the gradients in ``grads`` (see ``binding.AdamW.step``)."""
        self.optimizer.step(lr, step, **kw)

    @staticmethod
    def _chunk_buffer(t, s, e):
        """Rows [s, e) of t as one dense tensor: in place for one sequence, else a temporary."""
        v = t[:, s:e]
        return v if v.is_contiguous() else torch.empty(v.shape, dtype=t.dtype, device=t.device)

    @staticmethod
    def _keep(part, whole, s, e):
        if part.data_ptr() != whole[:, s:e].data_ptr():
            whole[:, s:e].copy_(part)
