"""Batches of matrices, (batch, rows, cols), that between them are made by every
kernel for products that the Muon calls choose: each role with each tile.  The
choice goes by a time model, so test_muon_cases_cpu.py asks the library for it."""
import ctypes as C

from memory_compressed_adaptive_amd import _lib as L

CASES = [
    (1, 130, 1223), (1, 130, 129), (3, 100, 5461), (4, 4098, 100), (13, 6340, 220), (64, 11540, 75),
    (138, 130, 296), (139, 131, 180), (168, 223, 130), (32, 696, 1405), (8, 2289, 1442),
    (1, 2048, 8192), (1, 4096, 11008), (1, 11008, 4096),
    # more than one run of matrices through the workspace, the last one shorter
    (71, 900, 899), (53, 1024, 1024), (89, 640, 1601), (83, 1700, 650),
]


def plan(batch, rows, cols):
    out = (C.c_int64 * 9)()
    L.check(L.lib().ma_debug_muon_plan(batch, rows, cols, out))
    names = ("small", "tall", "chunk", "pairs", "gram", "parts", "poly", "update", "last")
    return dict(zip(names, out))


def kernels(batch, rows, cols):
    """{(role, tile)} of the products of five steps; none where one workgroup takes a matrix."""
    p = plan(batch, rows, cols)
    if p["small"]:
        return set()
    made = {("X Xt in parts" if p["parts"] > 1 else "X Xt", p["gram"]), ("P", p["poly"]), ("P X", p["update"]),
            ("last, tall" if p["tall"] else "last", p["last"])}
    return made | ({("of two steps", p["poly"])} if p["pairs"] else set())


def runs(batch, rows, cols):
    """First and last matrix of every run through the workspace."""
    chunk = plan(batch, rows, cols)["chunk"] or batch
    return [(at, min(at + chunk, batch) - 1) for at in range(0, batch, chunk)]
