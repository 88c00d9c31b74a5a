"""AdamW over all of a model's tensors in one launch (a launch per 400), with
moments in fp32 or in 8-bit blocks."""
from __future__ import annotations

import torch

from . import AMSIM_ADAMW_BLOCK, AdamwTensor, adamw_moment_values, adamw_step, adamw_table


class AdamW(torch.optim.Optimizer):
    """AdamW with decoupled weight decay.

    fp32 parameters are updated in place.  bf16 parameters (VocabHead's weight)
    keep an fp32 master in the state, which is updated; the step writes its
    rounding to the parameter.  Gradients may be fp32 or bf16.
    moment_bits: 32, or 8 (one byte per moment and element and an fp32 scale
    per 256 of them).  grad_scale given to step() is one fp32 CUDA value that
    multiplies every gradient, such as the factor of clipping by the norm;
    reading it costs no synchronisation.
    """

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 moment_bits: int = 32):
        if moment_bits not in (8, 32):
            raise ValueError("moment_bits is 8 or 32")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay,
                                      moment_bits=moment_bits, step=0))
        self._tables = {}

    def _state(self, p, bits):
        st = self.state[p]
        if st:
            return st
        n = p.numel()
        if bits == 32:
            st["m"], st["v"] = (torch.zeros(n, dtype=torch.float32, device=p.device) for _ in range(2))
        else:
            st["m"] = torch.zeros(n, dtype=torch.int8, device=p.device)
            st["v"] = torch.zeros(n, dtype=torch.uint8, device=p.device)
            blocks = -(-n // AMSIM_ADAMW_BLOCK)
            st["m_scale"], st["v_scale"] = (torch.zeros(blocks, dtype=torch.float32, device=p.device) for _ in range(2))
        if p.dtype == torch.bfloat16:
            st["master"] = p.detach().float().reshape(-1)
        return st

    def _table(self, index, group):
        """The group's table; built again only when an address in it changed."""
        entries, key = [], []
        for p in group["params"]:
            if p.grad is None or p.numel() == 0:
                continue
            if p.dtype not in (torch.float32, torch.bfloat16):
                raise TypeError("AdamW takes fp32 and bf16 parameters")
            if not p.is_contiguous() or p.grad.is_sparse:
                raise ValueError("AdamW takes contiguous parameters with dense gradients")
            g = p.grad if p.grad.is_contiguous() else p.grad.contiguous()
            st = self._state(p, group["moment_bits"])
            entries.append((p, g, st))
            key.append((p.data_ptr(), p.numel(), g.data_ptr(), g.dtype, *[t.data_ptr() for t in st.values()]))
        key = (tuple(key), group["weight_decay"])
        kept = self._tables.get(index)
        if kept is not None and kept[0] == key:
            return kept[1], [g for _, g, _ in entries]
        table = adamw_table(
            AdamwTensor.make(st.get("master", p.detach().reshape(-1)), g.reshape(-1), st["m"], st["v"],
                             m_scale=st.get("m_scale"), v_scale=st.get("v_scale"),
                             copy=p.detach().reshape(-1) if "master" in st else None,
                             weight_decay=group["weight_decay"]) for p, g, st in entries)
        self._tables[index] = (key, table)
        return table, [g for _, g, _ in entries]

    @torch.no_grad()
    def step(self, closure=None, *, grad_scale: torch.Tensor | None = None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for i, group in enumerate(self.param_groups):
            table, hold = self._table(i, group)
            group["step"] += 1
            if len(table):
                adamw_step(table, lr=group["lr"], beta1=group["betas"][0], beta2=group["betas"][1], eps=group["eps"],
                           step=group["step"], grad_scale=grad_scale)
            del hold                     # gradients made contiguous live until the launch
        return loss

    def moments(self, p):
        """(first, second) moments of a parameter as fp32 values in its shape (a checkpoint's view of them)."""
        st = self.state[p]
        if "m_scale" not in st:
            return st["m"].view(p.shape), st["v"].view(p.shape)
        return (adamw_moment_values(st["m"], st["m_scale"]).view(p.shape),
                adamw_moment_values(st["v"], st["v_scale"]).view(p.shape))

    def load_state_dict(self, state_dict):
        """As torch's, but the state keeps its own types (torch would cast it to the parameter's)."""
        super().load_state_dict(state_dict)
        saved = state_dict["state"]
        order = [p for g in self.param_groups for p in g["params"]]
        for index, st in saved.items():
            for name, t in st.items():
                self.state[order[index]][name] = t.detach().clone().to(order[index].device)
        self._tables = {}
