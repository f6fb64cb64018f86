"""Trees of drafted tokens over a pool of states, and the pool's slots: the binding of their
entry points. As in ``kda``, every call marshals its arguments and runs the library; index
tensors live on the device and nothing waits for it."""
from __future__ import annotations

from typing import Optional

import torch

from .kda import (_FLOAT_IO, KDAError, _at, _dt, _expect, _expect_workspace, _options, _running, _same_gpu, _stream,
                  _workspace, load_library)
from .linear import _gate

_F32, _I32 = (torch.float32,), (torch.int32,)


def _tree_shapes(k, v, S, slot_in, parent, lin):
    """Checks what outputs and accepted states share; returns (N, T, H, Hk, Dk, Dv)."""
    for name, x in (("k", k), ("v", v)):
        if not isinstance(x, torch.Tensor) or x.dim() != 4:
            raise ValueError(f"{name} must be a 4-D tensor [N, T, heads, channels]")
    N, T, Hk, Dk = k.shape
    H, Dv = v.shape[2:]
    _expect(k, "k", (N, T, Hk if lin else H, Dk), _FLOAT_IO)
    _expect(v, "v", (N, T, H, Dv), (k.dtype,))
    if not isinstance(S, torch.Tensor) or S.dim() != 4:
        raise ValueError("S must be a pool of states [slots, H, Dv, Dk]")
    _expect(S, "S", (S.shape[0], H, Dv, Dk), _F32)
    _expect(slot_in, "slot_in", (N,), _I32, optional=True)
    _expect(parent, "parent", (N, T), _I32)
    return N, T, H, Hk, Dk, Dv


def _delta_gate(g, beta, N, T, H, Dk, head):
    if head:
        _expect(g, "g", (N, T, H), _F32, optional=True)
    else:
        _expect(g, "g", (N, T, H, Dk), _F32)
    _expect(beta, "beta", (N, T, H), _FLOAT_IO)


def _tree(entry, q, k, v, g, beta, S, slot_in, parent, out, out_dtype, stream, qk_l2norm=False, l2norm_eps=1e-6):
    lib = load_library()
    lin, head = entry == "lin_tree", entry == "gdn_tree"
    N, T, H, Hk, Dk, Dv = _tree_shapes(k, v, S, slot_in, parent, lin)
    _expect(q, "q", k.shape, (k.dtype,))
    if lin:
        gate = _gate(g, (N, T), H)
    else:
        _delta_gate(g, beta, N, T, H, Dk, head)
    _expect(out, "out", v.shape, _FLOAT_IO, optional=True)
    dev = _same_gpu(q=q, k=k, v=v, g=g, beta=beta, S=S, slot_in=slot_in, parent=parent, out=out)
    zero_rows = int(out is None)        # rows of absent nodes: left alone in the caller's out
    with _running(dev, stream):
        if out is None:
            out = torch.empty(v.shape, dtype=out_dtype or v.dtype, device=dev)
        if lin:
            st = lib.lin_tree(_at(q), _at(k), _at(v), _at(g), _at(S), _at(out), _at(slot_in), _at(parent), N, T, H, Hk, Dk, Dv,
                              S.shape[0], _dt(q), _dt(out), gate, zero_rows, _stream(stream, dev))
        else:
            st = lib.kda_tree(_at(q), _at(k), _at(v), _at(g), _at(beta), _at(S), _at(out), _at(slot_in), _at(parent), N, T, H,
                              Dk, Dv, S.shape[0], _dt(q), _dt(beta), _dt(out), zero_rows,
                              _options(head, qk_l2norm, l2norm_eps), _stream(stream, dev))
    if st != 0:
        raise KDAError(st, entry)
    return out


def kda_tree(q, k, v, g, beta, S, slot_in, parent, *, out=None, out_dtype: Optional[torch.dtype] = None, stream=None,
             qk_l2norm: bool = False, l2norm_eps: float = 1e-6):
    """The outputs of a tree of up to 64 drafted tokens that continues each sequence's state; no state is
    written. q, k, g: [N, T, H, Dk]; v: [N, T, H, Dv]; beta: [N, T, H]; S: [slots, H, Dv, Dk] fp32, slot_in
    (int32 [N], or None) each sequence's slot, negative = the zero state. parent: int32 [N, T], an earlier
    node, or -1 for the sequence's own state; with any other value the node is absent, with all that
    descend from it. Returns out [N, T, H, Dv]; rows of absent nodes are zero, but left as they were
    in an ``out`` that is given."""
    return _tree("kda_tree", q, k, v, g, beta, S, slot_in, parent, out, out_dtype, stream, qk_l2norm, l2norm_eps)


def gdn_tree(q, k, v, g, beta, S, slot_in, parent, *, out=None, out_dtype: Optional[torch.dtype] = None, stream=None,
             qk_l2norm: bool = False, l2norm_eps: float = 1e-6):
    """kda_tree with the scalar gate of Gated DeltaNet: g [N, T, H] fp32, or None for DeltaNet (no decay)."""
    return _tree("gdn_tree", q, k, v, g, beta, S, slot_in, parent, out, out_dtype, stream, qk_l2norm, l2norm_eps)


def lin_tree(q, k, v, g, S, slot_in, parent, *, out=None, out_dtype: Optional[torch.dtype] = None, stream=None):
    """kda_tree for linear attention without the delta rule: q, k [N, T, Hk, Dk], g [N, T, H] or [H] fp32, or None."""
    return _tree("lin_tree", q, k, v, g, None, S, slot_in, parent, out, out_dtype, stream)


def _accept(entry, k, v, g, beta, S, slot_in, slot_out, parent, node, stream, k_l2norm=False, l2norm_eps=1e-6):
    lib = load_library()
    lin, head = entry == "lin_tree_accept", entry == "gdn_tree_accept"
    N, T, H, Hk, Dk, Dv = _tree_shapes(k, v, S, slot_in, parent, lin)
    if lin:
        gate = _gate(g, (N, T), H)
    else:
        _delta_gate(g, beta, N, T, H, Dk, head)
    _expect(slot_out, "slot_out", (N,), _I32)
    _expect(node, "node", (N,), _I32)
    dev = _same_gpu(k=k, v=v, g=g, beta=beta, S=S, slot_in=slot_in, slot_out=slot_out, parent=parent, node=node)
    with _running(dev, stream):
        if lin:
            st = lib.lin_tree_accept(_at(k), _at(v), _at(g), _at(S), _at(slot_in), _at(slot_out), _at(parent), _at(node), N, T,
                                     H, Hk, Dk, Dv, S.shape[0], _dt(k), gate, _stream(stream, dev))
        else:
            st = lib.kda_tree_accept(_at(k), _at(v), _at(g), _at(beta), _at(S), _at(slot_in), _at(slot_out), _at(parent),
                                     _at(node), N, T, H, Dk, Dv, S.shape[0], _dt(k), _dt(beta),
                                     _options(head, k_l2norm, l2norm_eps), _stream(stream, dev))
    if st != 0:
        raise KDAError(st, entry)


def kda_tree_accept(k, v, g, beta, S, slot_in, slot_out, parent, node, *, stream=None, k_l2norm: bool = False,
                    l2norm_eps: float = 1e-6):
    """The state behind node[n] (int32 [N]; -1: the sequence's own state) of a tree as kda_tree takes it, into slot
    slot_out[n] (int32 [N]; negative: none) of the pool S. It may be the sequence's own slot; a slot that one
    sequence writes must not be read nor written by another one of the call. A node that is absent or out of
    range writes nothing."""
    _accept("kda_tree_accept", k, v, g, beta, S, slot_in, slot_out, parent, node, stream, k_l2norm, l2norm_eps)


def gdn_tree_accept(k, v, g, beta, S, slot_in, slot_out, parent, node, *, stream=None, k_l2norm: bool = False,
                    l2norm_eps: float = 1e-6):
    """kda_tree_accept with the scalar gate of Gated DeltaNet: g [N, T, H] fp32, or None for DeltaNet."""
    _accept("gdn_tree_accept", k, v, g, beta, S, slot_in, slot_out, parent, node, stream, k_l2norm, l2norm_eps)


def lin_tree_accept(k, v, g, S, slot_in, slot_out, parent, node, *, stream=None):
    """kda_tree_accept for linear attention without the delta rule: k [N, T, Hk, Dk], g [N, T, H] or [H], or None."""
    _accept("lin_tree_accept", k, v, g, None, S, slot_in, slot_out, parent, node, stream)


# ---- slots ------------------------------------------------------------------

def _pool(pool, name):
    """A pool of states: (layers, slots, bytes of a slot)."""
    if not isinstance(pool, torch.Tensor) or pool.dim() not in (4, 5):
        raise ValueError(f"{name} must be a pool of states [slots, H, Dv, Dk] or [layers, slots, H, Dv, Dk]")
    layers, slots = pool.shape[:2] if pool.dim() == 5 else (1, pool.shape[0])
    if pool.numel() == 0:
        raise ValueError(f"{name} is empty")
    return layers, slots, pool.numel() // (layers * slots) * pool.element_size()


def _few(x, name):
    """The library counts entries in 32 bits."""
    if x.numel() >= 2 ** 30:
        raise ValueError(f"{name} must have fewer than 2^30 entries")


def _counts(uses):
    if not isinstance(uses, torch.Tensor) or uses.dim() != 1 or uses.numel() == 0:
        raise ValueError("uses must be a 1-D tensor of counts, one per slot")
    _few(uses, "uses")
    _expect(uses, "uses", uses.shape, _I32)


def _indices(x, name):
    if not isinstance(x, torch.Tensor) or x.dim() != 1:
        raise ValueError(f"{name} must be a 1-D tensor")
    _expect(x, name, x.shape, _I32)
    _few(x, name)


def kda_slots_copy(pool, src, dst, *, to=None, stream=None):
    """Copies states between slots, in every layer: slot dst[i] becomes slot src[i] (int32 [n] each). pool:
    [slots, H, Dv, Dk] or [layers, slots, H, Dv, Dk]; ``to``: another pool for the copies, of the same
    layers and states (None: the same pool, a fork). A negative src: the zero state; a negative dst: nothing.
    A slot that is written must not be read nor written again by another entry."""
    lib = load_library()
    layers, slots, size = _pool(pool, "pool")
    _indices(src, "src")
    _expect(dst, "dst", src.shape, _I32)
    into = pool if to is None else to
    to_layers, to_slots, to_size = _pool(into, "to")
    if (to_layers, to_size, into.dtype) != (layers, size, pool.dtype):
        raise ValueError("to must have pool's dtype, layers and states")
    dev = _same_gpu(pool=pool, src=src, dst=dst, to=to)
    with _running(dev, stream):
        st = lib.kda_slots_copy(_at(pool), _at(into), _at(src), _at(dst), src.numel(), layers, slots, to_slots, size,
                                _stream(stream, dev))
    if st != 0:
        raise KDAError(st, "kda_slots_copy")


def _count(entry, uses, which, stream):
    lib = load_library()
    _counts(uses)
    _indices(which, "which")
    dev = _same_gpu(uses=uses, which=which)
    with _running(dev, stream):
        st = getattr(lib, entry)(_at(uses), _at(which), which.numel(), uses.numel(), _stream(stream, dev))
    if st != 0:
        raise KDAError(st, entry)


def kda_slots_share(uses, which, *, stream=None):
    """One use more for every slot in ``which`` (int32 [n]; a slot named twice counts twice; entries outside the
    pool are skipped). uses: int32 [slots], 0 = free."""
    _count("kda_slots_share", uses, which, stream)


def kda_slots_release(uses, which, *, stream=None):
    """One use less for every slot in ``which``; a count stays at zero."""
    _count("kda_slots_release", uses, which, stream)


def kda_slots_acquire(uses, n: int, *, taken=None, stream=None):
    """Takes the n lowest free slots, whose uses become 1. Returns them, int32 [n] ascending, -1 where there are no more."""
    lib = load_library()
    _counts(uses)
    if not isinstance(n, int) or not 0 <= n < 2 ** 30:
        raise ValueError("n must be a count of slots")
    _expect(taken, "taken", (n,), _I32, optional=True)
    dev = _same_gpu(uses=uses, taken=taken)
    with _running(dev, stream):
        if taken is None:
            taken = torch.empty(n, dtype=torch.int32, device=dev)
        st = lib.kda_slots_acquire(_at(uses), _at(taken), n, uses.numel(), _stream(stream, dev))
    if st != 0:
        raise KDAError(st, "kda_slots_acquire")
    return taken


def kda_slots_compact(pool, uses, table=None, *, count=None, workspace=None, stream=None):
    """Moves the pool's live slots to its front: with c slots in use, those at or behind c go, in ascending order,
    to the free ones before c, in every layer and in ``uses``. table (int32, any shape, or None): slot
    numbers, rewritten in place to where the slots went (-1: it was free; entries outside the pool stay).
    Returns c as an int32 tensor [1]."""
    lib = load_library()
    layers, slots, size = _pool(pool, "pool")
    _counts(uses)
    _expect(uses, "uses", (slots,), _I32)
    if table is not None:
        _expect(table, "table", getattr(table, "shape", None), _I32)
        _few(table, "table")
    _expect(count, "count", (1,), _I32, optional=True)
    _expect_workspace(workspace)
    dev = _same_gpu(pool=pool, uses=uses, table=table, count=count, workspace=workspace)
    with _running(dev, stream):
        if count is None:
            count = torch.empty(1, dtype=torch.int32, device=dev)
        workspace, ws_bytes = _workspace(int(lib.kda_slots_compact_workspace_size(slots)), workspace, dev)
        st = lib.kda_slots_compact(_at(pool), _at(uses), _at(table), _at(count), 0 if table is None else table.numel(), layers,
                                   slots, size, _at(workspace), ws_bytes, _stream(stream, dev))
    if st != 0:
        raise KDAError(st, "kda_slots_compact")
    return count
