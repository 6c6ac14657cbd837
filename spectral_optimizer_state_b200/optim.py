"""Muon for the selected projection weights, AdamW for everything else.

The protocol of "Muon Meets Mamba: Spectral Optimization for State Space
Models" (abstract) trains Mamba-2 130M with Muon on the output projections
only, the input projections only, or both, and AdamW for the rest; the
practitioner notes on the same paper (section 3.3) split the parameters by
name.  This class is the host-side bookkeeping of that split: parameters are
grouped by shape and dtype and handed to libmuon's muon_step_groups (Muon)
and muon_adamw_step (AdamW); every update runs in the library's kernels.
"""
from __future__ import annotations

from collections import OrderedDict

from .binding import MAX_BATCH, MAX_GROUPS, Muon, adamw_step, check_block


def takes_muon(name: str, shape, mode: str = "both", stacked: bool = False) -> bool:
    """2-D weights whose name marks them as the selected projection group(s); with ``stacked`` also
    3-D stacks of them (experts x rows x cols)."""
    if len(shape) != 2 and not (stacked and len(shape) == 3):
        return False
    if mode == "both":
        return "in_proj" in name or "out_proj" in name
    if mode in ("in_proj", "out_proj"):
        return mode in name
    if mode == "none":
        return False
    raise ValueError(f"unknown Muon selection {mode!r}")


class MuonAdamW:
    """named_params: iterable of (name, tensor) on one CUDA device.

    stacked: also give Muon the 3-D parameters whose name selects them, stacks of per-expert
    matrices (experts x rows x cols); every matrix is stepped on its own.
    blocks: {part of a name: (block rows, block cols)}; a selected parameter whose name contains the
    part is stepped block by block (``Muon.step_blocks``: heads of a projection, small experts), the
    first match counting.  None in place of a size means the whole side.  A block that ``Muon.step_blocks``
    does not take is refused here.
    """

    def __init__(self, named_params, mode="both", device=0, coeffs=None,
                 muon_hp=None, adamw_hp=None, stacked=False, blocks=None):
        import torch
        self.mode = mode
        self.muon_hp = dict(lr=0.02, beta=0.95, weight_decay=0.1, eps=1e-7, nesterov=True)
        self.muon_hp.update(muon_hp or {})
        self.adamw_hp = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
        self.adamw_hp.update(adamw_hp or {})
        named_params = [(name, p) for name, p in named_params]
        cut = {}  # name -> block of the parameters that are stepped block by block
        for name, p in named_params:
            block = next((tuple(b) for part, b in (blocks or {}).items() if part in name), None)
            if block is not None and takes_muon(name, tuple(p.shape), mode, stacked):
                check_block(p.shape[-2:], block, p.dtype)
                cut[name] = block
        self.ctx = Muon(device, coeffs)
        self.muon = OrderedDict()   # (shape, dtype[, block]) -> [(name, W, M)]
        self.adam = OrderedDict()   # dtype -> [(name, W, m, v)]
        for name, p in named_params:
            if takes_muon(name, tuple(p.shape), mode, stacked):
                key = (tuple(p.shape), p.dtype)
                if name in cut:
                    key += (cut[name],)
                self.muon.setdefault(key, []).append((name, p, torch.zeros(p.shape, dtype=torch.float32, device=p.device)))
            else:
                z = lambda: torch.zeros(p.numel(), dtype=torch.float32, device=p.device)  # noqa: E731
                self.adam.setdefault(p.dtype, []).append((name, p, z(), z()))
        self.t = 0
        # AdamW bias correction counts the steps each parameter actually took (a parameter
        # without a gradient in some step keeps its count, as in torch.optim.AdamW)
        self.adam_t = {n: 0 for entries in self.adam.values() for (n, _, _, _) in entries}

    def muon_names(self):
        return [n for entries in self.muon.values() for (n, _, _) in entries]

    def adamw_names(self):
        return [n for entries in self.adam.values() for (n, _, _, _) in entries]

    @staticmethod
    def _gradient(w, g, stream):
        """g as the kernels read it: of w's dtype (rounded on `stream` if it is of another) and contiguous."""
        if g.dtype == w.dtype and g.is_contiguous():
            return g
        if stream is None:
            return g.to(w.dtype).contiguous()
        import torch
        with torch.cuda.stream(stream):
            return g.to(w.dtype).contiguous()

    def step(self, grads, stream=None):
        """grads: mapping name -> gradient tensor of the parameter's shape.  One of another dtype (the fp32
        buffer that micro-batches of bf16 weights were accumulated in) is rounded to the parameter's first.

        A parameter whose name is missing from ``grads`` or maps to None (frozen, or unused
        in this backward pass) is left untouched: its weights get no decay, its Muon momentum
        no step and its AdamW moments and step count stay as they are.

        ``ctx.status()`` afterwards covers every block of the step, and the whole matrices of its last call
        (of up to MAX_GROUPS groups).
        """
        self.t += 1
        groups = []
        for key, entries in self.muon.items():
            live = [(w, self._gradient(w, grads[n], stream), mbuf) for n, w, mbuf in entries if grads.get(n) is not None]
            if len(key[0]) == 3:  # a stack: its matrices one by one
                live = [t for w, g, mbuf in live for t in zip(w.unbind(0), g.unbind(0), mbuf.unbind(0))]
            for c0 in range(0, len(live), MAX_BATCH):
                chunk = tuple(list(ts) for ts in zip(*live[c0:c0 + MAX_BATCH]))
                if len(key) == 3:
                    self.ctx.step_blocks(*chunk, key[2], stream=stream, **self.muon_hp)
                else:
                    groups.append(chunk)
        for g0 in range(0, len(groups), MAX_GROUPS):
            self.ctx.step_groups(groups[g0:g0 + MAX_GROUPS], stream=stream, **self.muon_hp)
        for entries in self.adam.values():
            by_count = OrderedDict()  # one launch per distinct step count (normally exactly one)
            for e in entries:
                if grads.get(e[0]) is None:
                    continue
                self.adam_t[e[0]] += 1
                by_count.setdefault(self.adam_t[e[0]], []).append(e)
            for t, live in by_count.items():
                W = [w.view(-1) for _, w, _, _ in live]
                G = [self._gradient(w, grads[n], stream).view(-1) for n, w, _, _ in live]
                adamw_step(W, G, [m for _, _, m, _ in live], [v for _, _, _, v in live], t,
                           stream=stream, **self.adamw_hp)

    def state_dict(self) -> dict:
        """Optimizer state by parameter name: Muon momentum, AdamW moments, and the step count."""
        return {"t": self.t, "adamw_t": dict(self.adam_t),
                "muon": {n: m.detach().clone() for entries in self.muon.values() for (n, _, m) in entries},
                "adamw": {n: (m.detach().clone(), v.detach().clone())
                          for entries in self.adam.values() for (n, _, m, v) in entries}}

    def load_state_dict(self, state: dict):
        """Restore the state saved by ``state_dict`` for the same parameter names and shapes."""
        muon = {n: m for entries in self.muon.values() for (n, _, m) in entries}
        adam = {n: (m, v) for entries in self.adam.values() for (n, _, m, v) in entries}
        if set(state["muon"]) != set(muon) or set(state["adamw"]) != set(adam):
            raise ValueError("checkpoint holds a different parameter split")
        for n, m in state["muon"].items():
            muon[n].copy_(m)
        for n, (m, v) in state["adamw"].items():
            adam[n][0].copy_(m)
            adam[n][1].copy_(v)
        self.t = int(state["t"])
        counts = state.get("adamw_t", {n: self.t for n in adam})
        self.adam_t = {n: int(counts[n]) for n in adam}

    def close(self):
        self.ctx.close()


def torch_optimizer(named_params, mode="both", inner=None, main_grads=None, **kw):
    """A ``torch.optim.Optimizer`` over MuonAdamW: ``step()`` reads each parameter's ``.grad``.

    named_params: (name, parameter) pairs, e.g. ``model.named_parameters()``.  Parameters whose
    ``.grad`` is None at ``step()`` are skipped, as ``torch.optim.AdamW`` skips them: no decay,
    no momentum step, no moment update.  ``main_grads`` ({name: buffer}) names the parameters whose
    gradients are accumulated elsewhere (``expert_linear(..., grad_into=buffer)``, which leaves ``.grad``
    None): ``step()`` reads their buffers and ``zero_grad()`` clears them.  ``inner`` replaces the
    MuonAdamW instance (host-side tests only).
    """
    import torch

    named = [(n, p) for n, p in named_params]
    buffers = dict(main_grads or {})
    shapes = {n: p.shape for n, p in named}
    for n, b in buffers.items():
        if n not in shapes or b.shape != shapes[n]:
            raise ValueError(f"main_grads: {n} is no parameter of shape {tuple(b.shape)}")

    class MuonAdamWOptimizer(torch.optim.Optimizer):
        def __init__(self):
            super().__init__([p for _, p in named], defaults={})
            self.inner = inner if inner is not None else MuonAdamW(named, mode=mode, **kw)
            self.names = [n for n, _ in named]

        @torch.no_grad()
        def step(self, closure=None):
            loss = None
            if closure is not None:
                with torch.enable_grad():
                    loss = closure()
            for n, p in named:
                if n in buffers and p.grad is not None:
                    raise ValueError(f"{n} has both a gradient and an accumulation buffer")
            grads = {n: buffers.get(n, p.grad) for n, p in named}
            self.inner.step(grads)
            return loss

        def zero_grad(self, set_to_none=True):
            super().zero_grad(set_to_none)
            for b in buffers.values():
                b.zero_()

        def state_dict(self):
            return self.inner.state_dict()

        def load_state_dict(self, state):
            self.inner.load_state_dict(state)

    return MuonAdamWOptimizer()
