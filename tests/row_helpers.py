"""What the tests of the row operators share: rows in device storage with a
marker around them, and comparisons with a tolerance for every element."""
import numpy as np
import torch

U = 2.0 ** -24                            # half a step of fp32
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = {"f32": 1e-37, "bf16": 1e-37}      # below the smallest normal number nothing is promised


def torch_type(dtype):
    return torch.float32 if dtype == "f32" else torch.bfloat16


class Rows:
    """[M, C] values (or zeros) of a type in rows `ld` apart, `skip` elements into their storage, a marker elsewhere."""

    def __init__(self, M, C, dtype, values=None, pad=0, skip=0, marker=7.0, device="cuda"):
        self.ld, self.M, self.C, self.skip, self.marker = C + pad, M, C, skip, marker
        self.type = torch_type(dtype) if isinstance(dtype, str) else dtype
        self.store = torch.full((skip + M * self.ld + 64,), marker, dtype=self.type, device=device)
        self.view = self.store[skip:skip + M * self.ld].view(M, self.ld)[:, :C]
        if values is not None:
            self.view.copy_(torch.as_tensor(values))

    def data_ptr(self):
        return self.view.data_ptr()

    def host(self):
        return self.view.double().cpu().numpy()

    def untouched(self):
        s = self.store.clone()
        s[self.skip:self.skip + self.M * self.ld].view(self.M, self.ld)[:, :self.C] = self.marker
        return bool((s == self.marker).all().item())


def inside(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = int(np.flatnonzero(bad.reshape(-1))[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; first {i}: got {got.reshape(-1)[i]!r} want "
                             f"{want.reshape(-1)[i]!r} tol {np.broadcast_to(tol, want.shape).reshape(-1)[i]!r}")
