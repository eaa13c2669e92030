"""One Orthros attention layer with rotary positions, made of the library's calls.

The pages leave the positional encoding aside; a model with rotary positions
turns queries and keys between the stream affines and the attention (Alg. 1
lines 5 and 7). `RotaryLayer` shows where those calls stand:

serving   step(): projection -> rotated paged append -> attention of the new
          tokens over the cache, base stream (window) and output stream (all
          keys). One token per sequence, chunks of prompts, or both mixed; no
          length is read on the host, so a step can be captured in a CUDA graph.
training  forward() / backward(): rotation of affined queries and of keys ->
          orthros_prefill with identity affines, and the gradients back through
          both, those of the four affines included.
"""
from __future__ import annotations

import dataclasses

import torch

from . import _binding as ops


def _add_rows(x, rows, y):
    """x[rows[i]] += y[i] in place, in fp32 and rounded once per row of x. Rows may repeat: the y of a
    row are summed in the order they stand in (an indexed add with atomics would take any order, and
    through an fp32 copy of x it would move all of x for a few rows)."""
    if rows.numel() == 0:
        return
    rows, order = torch.sort(rows, stable=True)
    run = torch.zeros_like(rows)  # which run of equal rows an entry belongs to
    run[1:] = (rows[1:] != rows[:-1]).cumsum(0)
    total = torch.zeros(y.shape, dtype=torch.float32, device=y.device)
    total.index_put_((run,), y[order].float(), accumulate=True)  # (sorts its indices, no atomics)
    x[rows] = (x[rows].float() + total[run]).to(x.dtype)  # entries of a run write the same value


@dataclasses.dataclass
class RotaryLayer:
    """Weights and shape of the layer. `affines` are alpha_base, beta_base, alpha_out,
    beta_out [Hq, d]; `freq` [rot_dim/2] the rotary frequencies (orthros_rotary_frequencies)."""

    w_qkv: torch.Tensor  # [(Hq + 2 Hkv) d, d_model] bf16
    affines: list
    freq: torch.Tensor
    Hq: int
    Hkv: int
    d: int
    window: int
    layout: str = "half"
    amplitude: float = 1.0

    def __post_init__(self):
        dev = self.w_qkv.device
        self.steps = ops.orthros_rotary_steps(self.freq).to(dev)
        self.identity = (torch.ones(self.Hq, self.d, device=dev), torch.zeros(self.Hq, self.d, device=dev))
        self._reports = []  # buffers that begin with a status word of the last step(), or forward() and backward()

    def _rope(self):
        return dict(layout=self.layout, amplitude=self.amplitude)

    def check(self, stream=None):
        """Synchronises `stream` (default: the current one) and returns (status, bits) of the last
        step(), or of the last forward() with the backward() after it: the first status that is not
        0 (orthros_check) and the ORTHROS_DEV_* bits of all its calls."""
        found = [ops.orthros_check(w, stream) for w in self._reports]
        bits = 0
        for _, b in found:
            bits |= b
        return next((s for s, _ in found if s), 0), bits

    # ---- serving -------------------------------------------------------------
    def step_workspaces(self, B, n_new, n_out, max_new, max_pages, page_size):
        """Workspaces of step() for these sizes or smaller ones: projection, append, both attentions."""
        sizes = [256, 256] + [ops.orthros_chunk_attention_workspace_size(B, n, m, self.Hq, self.Hkv, self.d, max_pages,
                                                                        page_size, self.w_qkv.dtype)
                              for n, m in ((n_new, max_new), (n_out, 1))]
        return [torch.empty(max(s, 256), dtype=torch.uint8, device=self.w_qkv.device) for s in sizes]

    def step(self, x, n_new, k_cache, v_cache, block_table, token_seq, token_pos, new_indptr, kv_lens, out_indptr,
             out_positions, max_new, workspaces=None):
        """One serving step.

        x [n_new + n_out, d_model]: the new tokens of the batch (rows new_indptr[b] ..
        new_indptr[b+1] belong to sequence b), then at most one output-stream token per
        sequence, at its last position (out_indptr, out_positions). kv_lens counts the
        cached tokens with the new ones. workspaces: step_workspaces(), kept by the caller, or None
        (allocated here; the layer holds them until its next step, for check()). A token whose
        sequence, position or page does not exist is not cached, which only check() tells.
        Returns (o_base [n_new, Hq, d], o_out [n_out, Hq, d]).
        """
        if workspaces is None:
            workspaces = self.step_workspaces(block_table.shape[0], n_new, x.shape[0] - n_new, max_new,
                                              block_table.shape[1], k_cache.shape[1])
        project, append, base, out = workspaces
        self._reports = []
        q, q_out, k, v = ops.orthros_qkv_project(x, n_new, self.w_qkv, self.Hq, self.Hkv, self.d, *self.affines,
                                                 kv_out=True, workspace=project)
        q, q_out = ops.orthros_rotate_append(q, k, v, k_cache, v_cache, block_table, token_seq, token_pos, self.steps,
                                             q_out=q_out, out_positions=out_positions, workspace=append, **self._rope())
        o_base, _ = ops.orthros_chunk_attention(q, new_indptr, kv_lens, k_cache, v_cache, block_table, self.window,
                                                max_new=max_new, workspace=base)
        o_out, _ = ops.orthros_chunk_attention(q_out, out_indptr, kv_lens, k_cache, v_cache, block_table, 2 ** 31 - 1,
                                               max_new=1, workspace=out)
        self._reports = [project, append, base, out]
        return o_base, o_out

    # ---- training ------------------------------------------------------------
    def forward(self, q, k, v, out_indptr, out_positions):
        """q [B, T, Hq, d] (before the affines), k, v [B, T, Hkv, d]; output rows as in
        orthros_prefill (their raw queries are q at their positions). A position outside
        [0, T) makes its output row NaN and has no gradient. Returns ((o_base, o_out), saved
        for backward)."""
        B, T = q.shape[:2]
        ab, bb, ao, bo = self.affines
        pos = torch.arange(T, dtype=torch.int32, device=q.device).repeat(B)
        counts = torch.as_tensor(out_indptr, dtype=torch.int64, device="cpu").diff()
        # (the prefill judges the positions; here they only have to stay within their sequence)
        rows = torch.repeat_interleave(torch.arange(B), counts).to(q.device) * T + out_positions.clamp(0, T - 1)
        qf, kf = q.flatten(0, 1), k.flatten(0, 1)
        q_sel = qf[rows]
        qr = ops.orthros_rotate(qf, pos, self.steps, alpha=ab, beta=bb, **self._rope()).view_as(q)
        kr = ops.orthros_rotate(kf, pos, self.steps, **self._rope()).view_as(k)
        qo = ops.orthros_rotate(q_sel, out_positions, self.steps, alpha=ao, beta=bo, **self._rope())
        need = ops.orthros_prefill_workspace_size(B, T, self.Hq, self.Hkv, self.d, qo.shape[0], self.window, q.dtype)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
        out = ops.orthros_prefill(qr, kr, v, *self.identity, *self.identity, out_indptr, out_positions, self.window,
                                  q_out=qo, workspace=ws)
        self._reports = [ws[:256].clone()]  # the status word; the scratch is not held
        return (out[0], out[2]), (qf, q_sel, rows, pos, qr, kr, v, qo, out_indptr, out_positions, out)

    def backward(self, saved, do_base, do_out):
        """Gradients of q, k, v and of the four affines, in a dict."""
        qf, q_sel, rows, pos, qr, kr, v, qo, out_indptr, out_positions, out = saved
        ab, _, ao, _ = self.affines
        need = ops.orthros_prefill_backward_workspace_size(*qr.shape[:2], self.Hq, self.Hkv, self.d, qo.shape[0],
                                                           self.window, qr.dtype)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=qr.device)
        g = ops.orthros_prefill_backward(qr, kr, v, *self.identity, *self.identity, out_indptr, out_positions,
                                         self.window, None, *out, do_base, do_out, q_out=qo, workspace=ws)
        self._reports = self._reports[:1] + [ws[:256].clone()]
        dq, da, db = ops.orthros_rotate_backward(g["dq"].flatten(0, 1), qf, pos, self.steps, alpha=ab, **self._rope())
        dk, _, _ = ops.orthros_rotate_backward(g["dk"].flatten(0, 1), None, pos, self.steps, affine_grads=False,
                                               **self._rope())
        outside = (out_positions < 0) | (out_positions >= qr.shape[1])  # rows that read nothing
        dq_out = g["dq_out"].masked_fill_(outside[:, None, None], 0)
        dq_sel, da_out, db_out = ops.orthros_rotate_backward(dq_out, q_sel, out_positions, self.steps, alpha=ao,
                                                             **self._rope())
        _add_rows(dq, rows, dq_sel)
        return {"dq": dq.view_as(qr), "dk": dk.view_as(kr), "dv": g["dv"], "d_alpha_base": da, "d_beta_base": db,
                "d_alpha_out": da_out, "d_beta_out": db_out}
