"""The gated delta rule through its C entry points, every output and the scratch,
of exactly the size asked for, between guards."""
import torch

import linear_recurrence_ssm_gb300 as lrs

GUARD = 4096        # bytes


class Guarded:
    """Tensors filled with 0xff (NaN in every type of the rule), GUARD bytes of 0x5a on either side of each."""

    def __init__(self, device):
        self.device, self.rooms = device, []

    def empty(self, *shape, dtype=torch.uint8):
        n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
        room = torch.full((GUARD + n + GUARD,), 0x5a, dtype=torch.uint8, device=self.device)
        room[GUARD:GUARD + n] = 0xff
        self.rooms.append(room)
        return room[GUARD:GUARD + n].view(dtype).view(shape)

    def untouched(self):
        return all((r[:GUARD] == 0x5a).all() and (r[-GUARD:] == 0x5a).all() for r in self.rooms)


def at(t):
    return None if t is None else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


def sizes(i, n):
    """Bs, L, G, H, K, V, n_seq, bf16 of the inputs, n: packed sequences or 0."""
    (Bs, L, G, K), (H, V) = i["q"].shape, i["v"].shape[2:]
    return Bs, L, G, H, K, V, n, int(i["v"].dtype is torch.bfloat16)


def forward(i, offsets=None, h0=None, scale=1.0, room=None):
    """(status, dict(y, h_final, states, errors)), all of them written into `room`."""
    room = room or Guarded(i["v"].device)
    n = 0 if offsets is None else offsets.numel() - 1
    Bs, L, G, H, K, V, _, bf16 = size = sizes(i, n)
    t, slots = i["v"].dtype, L // 64 + n if n else Bs * -(-L // 64)
    out = dict(y=room.empty(Bs, L, H, V, dtype=t), h_final=room.empty(n or Bs, H, V, K, dtype=torch.float32),
               states=room.empty(slots, H, V, K, dtype=t), errors=room.empty(Bs, L, H, V, dtype=t))
    scratch = room.empty(lrs.library().delta_rule_fwd_scratch(*size))
    status = lrs.library().delta_rule_fwd(*(at(i[w]) for w in ("q", "k", "v", "g", "beta")), scale, at(offsets), at(h0),
                                          *(at(w) for w in out.values()), at(scratch), *size, stream())
    return status, out


def backward(i, dy, kept, offsets=None, dh_final=None, scale=1.0, room=None):
    """(status, dict(dq, dk, dv, dg, dbeta, dh0))."""
    room = room or Guarded(dy.device)
    n = 0 if offsets is None else offsets.numel() - 1
    Bs, L, G, H, K, V, _, bf16 = size = sizes(i, n)
    t = dy.dtype
    out = dict(dq=room.empty(Bs, L, G, K, dtype=t), dk=room.empty(Bs, L, G, K, dtype=t),
               dv=room.empty(Bs, L, H, V, dtype=t), dg=room.empty(Bs, L, H, dtype=t),
               dbeta=room.empty(Bs, L, H, dtype=t), dh0=room.empty(n or Bs, H, V, K, dtype=torch.float32))
    scratch = room.empty(lrs.library().delta_rule_bwd_scratch(*size))
    status = lrs.library().delta_rule_bwd(*(at(i[w]) for w in ("q", "k", "g", "beta")), scale, at(offsets), at(dy),
                                          at(dh_final), at(kept["states"]), at(kept["errors"]),
                                          *(at(w) for w in out.values()), at(scratch), *size, stream())
    return status, out
