"""Calls the entry points of the operators around a verification step of a libsvd build
with arguments their host-side checks reject or only compute sizes from (fake, never
dereferenced addresses: no HIP call is reached), values outside the enumerators and at the
ends of the integer types included, and prints the status codes.  Run by
tests/test_abi_step_sanitized.py."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lossless_draft_verification_verifier_amd as svd  # noqa: E402

L = svd.Library(sys.argv[1])
I32, I64 = (1 << 31) - 1, (1 << 63) - 1
out = []


def cache(**kw):
    a = dict(k=4096, v=8192, k_scale=None, v_scale=None, block_table=12288, n_pages=10,
             max_pages=4, page=16, kv_heads=2, head_dim=64, dtype=svd.SVD_CACHE_BF16)
    a.update(kw)
    return svd.CacheStruct(*[a[n] for n, _ in svd.CacheStruct._fields_])


def write(c, **kw):
    a = dict(k=4096, v=8192, dtype=svd.SVD_BF16, ks=128, vs=128, ctx=64, B=2, T=3)
    a.update(kw)
    out.append(L.svd_cache_write(c, a["k"], a["v"], a["dtype"], a["ks"], a["vs"], a["ctx"], None,
                                 None, a["B"], a["T"], None))


def read(c, **kw):
    a = dict(B=2, N=3, dtype=svd.SVD_BF16, k=4096, v=8192)
    a.update(kw)
    out.append(L.svd_cache_read(c, None, None, a["B"], a["N"], a["dtype"], a["k"], a["v"], None))


def attend(c, **kw):
    a = dict(q=4096, qs=256, ctx=64, scale=0.125, B=2, T=3, Hq=4, out=1 << 16, ws=1 << 20, n=0)
    a.update(kw)
    out.append(L.svd_tree_attention(c, a["q"], a["qs"], a["ctx"], None, None, a["scale"], a["B"],
                                    a["T"], a["Hq"], a["out"], None, a["ws"], a["n"], None))


BAD = [dict(k=None), dict(dtype=2), dict(dtype=-5), dict(dtype=I32), dict(dtype=-I32 - 1),
       dict(dtype=1), dict(dtype=1, k_scale=65, v_scale=64), dict(head_dim=96),
       dict(head_dim=-I32), dict(page=48), dict(page=-I32 - 1), dict(page=0), dict(n_pages=I64),
       dict(n_pages=-1), dict(max_pages=I32), dict(max_pages=-1), dict(kv_heads=I32),
       dict(kv_heads=-1), dict(k=4100)]
for f in (write, read, attend):
    f(None)
    for kw in BAD:
        f(cache(**kw))
for kw in (dict(dtype=2), dict(dtype=I32), dict(ks=-I64), dict(vs=0), dict(k=4097), dict(B=0),
           dict(B=I64), dict(T=I64), dict(T=-I64), dict(B=1 << 30, T=1), dict(B=1, T=I32),
           dict(ctx=None)):
    write(cache(), **kw)
    if "ks" not in kw and "vs" not in kw and "ctx" not in kw:
        read(cache(), **{("N" if n == "T" else n): x for n, x in kw.items()})
for kw in (dict(), dict(B=I64), dict(B=1 << 29, T=1), dict(T=I32), dict(T=4096, B=1 << 17),
           dict(Hq=I32), dict(Hq=65536), dict(Hq=-4), dict(scale=3e38), dict(scale=float("nan")),
           dict(scale=1e-45), dict(qs=I64 - 7), dict(qs=-I64), dict(q=4104), dict(out=4096, n=I64),
           dict(ws=(1 << 20) + 8), dict(out=4096 + 512, n=1 << 40)):
    attend(cache(), **kw)
attend(cache(kv_heads=4096, max_pages=(1 << 27) - 1), Hq=65536, B=1 << 17, T=4096)
for args in ((1, 1, 32, 8, 128, 4096), (1, 1, 8, 8, 64, I32), (1 << 29, 1, 8, 8, 64, I32),
             (1, 4096, 65536, 1, 128, I32), (1 << 17, 4096, 65536, 4096, 128, I32),
             (I64, 4096, 8, 8, 64, 1), (1, 1, 8, 0, 64, 1), (1, 1, 8, 8, 64, I64),
             (-I64, 1, 8, 8, 64, 1), (1, -1, 8, 8, 64, 1), (1, 1, 8, 8, 64, -I64)):
    out.append(L.svd_tree_attention_workspace_bytes(*args))
for kw in (dict(d=None), dict(B=I64), dict(B=0), dict(K=I32), dict(K=-1), dict(G=I32), dict(T=I32),
           dict(T=-1), dict(B=1 << 29, T=2), dict(B=1 << 22, K=1, G=1, T=2)):
    a = dict(d=64, B=2, K=2, G=3, T=7)
    a.update(kw)
    out.append(L.svd_draft_tree(a["d"], None, a["B"], a["K"], a["G"], a["T"], 128, 192, 256, 320,
                                384, 448, None))
for kw in (dict(z=None), dict(dtype=2), dict(dtype=-I32), dict(B=I64), dict(T=I32), dict(V=-1),
           dict(hist=64), dict(hist=64, hlen=64, hs=I64), dict(anc=64), dict(boff=64, nb=-I64),
           dict(boff=64, nb=I64), dict(allow=64), dict(allow=64, ai=64, nm=-I32), dict(z=4097),
           dict(B=(1 << 30) - 1, T=1, V=I32), dict(B=1 << 17, T=4096, V=I32),
           dict(B=1 << 24, T=1, V=100)):
    a = dict(z=4096, out=8192, dtype=svd.SVD_BF16, B=2, T=3, V=100, hist=None, hs=0, hlen=None,
             tok=None, anc=None, boff=None, btok=None, bval=None, nb=0, allow=None, ai=None, nm=0)
    a.update(kw)
    out.append(L.svd_adjust_logits(a["z"], a["out"], a["dtype"], a["B"], a["T"], a["V"], None,
                                   a["hist"], a["hs"], a["hlen"], None, a["tok"], a["anc"], None,
                                   None, None, a["boff"], a["btok"], a["bval"], a["nb"],
                                   a["allow"], a["ai"], a["nm"], None))
assert svd.SVD_EHIP not in out and svd.SVD_OK not in out[:60], out
print(out)
