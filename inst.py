import sys, ctypes
sys.path.insert(0, ".")
import torch, numpy as np
from perf import operators as O
import kv_cache_retrieval_b200 as hhr
O.own = True
for n in sys.argv[1].split(","):
    c = [c for c in O.listed() if c["name"] == n][0]
    s = O.prepare(c, 0)
    for _ in range(3): O.run(s)
    buf = np.zeros((160, 8, 8), dtype=np.uint64)
    hhr.lib().hhr_dbg(ctypes.c_void_p(buf.ctypes.data))
    O.run(s); hhr.lib().hhr_dbg(ctypes.c_void_p(buf.ctypes.data))
    b = buf.astype(np.int64); on = b[..., 2] > 0
    t0 = b[..., 0][b[..., 0] > 0].min()
    f = lambda i: (b[..., i][on] - t0) / 1e3
    pc = lambda x: " ".join(f"{v:7.1f}" for v in np.percentile(x, [0, 10, 50, 90, 100]))
    print(n, "warps", on.sum(), "tiles/warp", b[..., 6][on].min(), b[..., 6][on].max())
    for i, k in ((0, "start"), (1, "prologue"), (2, "loop end"), (3, "cta end"), (4, "join end")): print("  %-9s" % k, pc(f(i)))
    u = b[..., 5][on]; e = f(2)
    print("  units/warp", pc(u), "corr(units, end)", np.corrcoef(u, e)[0, 1] if u.std() > 0 else None)
    for lo, hi in ((1, 1), (2, 2), (3, 4), (5, 8), (9, 99)):
        k = (u >= lo) & (u <= hi)
        if k.any(): print("   units %d-%d: %d warps, end %s" % (lo, hi, k.sum(), pc(e[k])))
    ce = (b[..., 2] - t0).max(1)[on.any(1)] / 1e3
    print("  cta ends", pc(ce))
