"""AdamW over all of a model's tensors in one launch (a launch per 400), with
moments in fp32 or in 8-bit blocks."""
from __future__ import annotations

import torch

from . import AMSIM_ADAMW_BLOCK, AdamwTensor, adamw_moment_values, adamw_step, adamw_table


class AdamW(torch.optim.Optimizer):
    """AdamW with decoupled weight decay.

    fp32 parameters are updated in place.  bf16 parameters (VocabHead's weight)
    keep an fp32 master in the state, which is updated; the step writes its
    rounding to the parameter.  Weights that are put into such a parameter (a
    module's load_state_dict, other memory given to p.data) go into its master
    before the next step; writes in place through .data are not seen.
    Gradients may be fp32 or bf16.
    moment_bits: 32, or 8 (one byte per moment and element and an fp32 scale
    per 256 of them).  Each parameter counts its own updates, by which its
    moments' bias is corrected; those with the same count share a launch.
    grad_scale given to step() is one fp32 CUDA value that multiplies every
    gradient, such as the factor of clipping by the norm; reading it costs no
    synchronisation.
    """

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 moment_bits: int = 32):
        if moment_bits not in (8, 32):
            raise ValueError("moment_bits is 8 or 32")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay,
                                      moment_bits=moment_bits))
        self._tables, self._versions = {}, {}

    def __setstate__(self, state):       # of a copy, whose tables are made at its first step
        super().__setstate__(state)
        self._tables, self._versions = {}, {}

    def _state(self, p, bits):
        if p.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("AdamW takes fp32 and bf16 parameters")
        n = p.numel()

        def zeros(count, dtype):
            return torch.zeros(count, dtype=dtype, device=p.device)
        if bits == 32:
            new = dict(m=zeros(n, torch.float32), v=zeros(n, torch.float32))
        else:
            blocks = -(-n // AMSIM_ADAMW_BLOCK)
            new = dict(m=zeros(n, torch.int8), v=zeros(n, torch.uint8), m_scale=zeros(blocks, torch.float32),
                       v_scale=zeros(blocks, torch.float32))
        if p.dtype == torch.bfloat16:
            new["master"] = p.detach().float().reshape(-1)
            self._versions[p] = p._version, p.data_ptr()
        st = self.state[p]
        st.update(new, step=0)
        return st

    def _follow(self, p, st):
        """The master takes the elements of a bf16 parameter that are no longer its rounding."""
        new, master = p.detach().reshape(-1), st["master"].view(-1)
        master.copy_(torch.where(master.to(new.dtype) == new, master, new.float()))
        self._versions[p] = p._version, p.data_ptr()

    def _group_tables(self, index, group):
        """The group's tables, one for each count of updates, as (count so far, table), and the gradients and states
        of their parameters.  Built again only when an address in them changed, or some counts against others.  (The
        loop is the host's time of a step: some 1.3 us a parameter.)"""
        entries, key, first, state = [], [group["weight_decay"]], None, self.state
        for p in group["params"]:
            g = p.grad
            if g is None or p.numel() == 0:
                continue
            if not p.is_contiguous() or g.is_sparse:
                raise ValueError("AdamW takes contiguous parameters with dense gradients")
            if not g.is_contiguous():
                g = g.contiguous()
            st = state[p] or self._state(p, group["moment_bits"])
            count = st["step"]
            if first is None:
                first = count
            entries.append((p, g, st))
            key += (p.data_ptr(), p.numel(), g.data_ptr(), g.dtype, count - first, st["m"].data_ptr(), st["v"].data_ptr())
            if "m_scale" in st:
                key += (st["m_scale"].data_ptr(), st["v_scale"].data_ptr())
            if "master" in st:
                if self._versions.get(p) != (p._version, p.data_ptr()):
                    self._follow(p, st)
                key.append(st["master"].data_ptr())
        kept = self._tables.get(index)
        if kept is None or kept[0] != key:
            by_count = {}
            for p, g, st in entries:
                by_count.setdefault(st["step"] - first, []).append(
                    AdamwTensor.make(st.get("master", p.detach().reshape(-1)), g.reshape(-1), st["m"], st["v"],
                                     m_scale=st.get("m_scale"), v_scale=st.get("v_scale"),
                                     copy=p.detach().reshape(-1) if "master" in st else None,
                                     weight_decay=group["weight_decay"]))
            kept = self._tables[index] = (key, [(ahead, adamw_table(es)) for ahead, es in by_count.items()])
        return [(first + ahead, table) for ahead, table in kept[1]], [g for _, g, _ in entries], [st for _, _, st in entries]

    @torch.no_grad()
    def step(self, closure=None, *, grad_scale: torch.Tensor | None = None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for i, group in enumerate(self.param_groups):
            tables, hold, states = self._group_tables(i, group)
            for count, table in tables:
                adamw_step(table, lr=group["lr"], beta1=group["betas"][0], beta2=group["betas"][1], eps=group["eps"],
                           step=count + 1, grad_scale=grad_scale)
            for st in states:
                st["step"] += 1
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
        """As torch's, but the state keeps its own types (torch would cast it to the parameter's).  A state that was
        saved with one count of updates for a group, not one for each parameter, goes on with that."""
        super().load_state_dict(state_dict)
        saved = state_dict["state"]
        order = [p for g in self.param_groups for p in g["params"]]
        for index, st in saved.items():
            for name, t in st.items():
                if isinstance(t, torch.Tensor):
                    self.state[order[index]][name] = t.detach().clone().to(order[index].device)
            self._versions[order[index]] = order[index]._version, order[index].data_ptr()    # the state has its master
        for group in self.param_groups:
            count = group.pop("step", None)
            for p in group["params"]:
                if count is not None and p in self.state:
                    self.state[p].setdefault("step", count)
        self._tables = {}
