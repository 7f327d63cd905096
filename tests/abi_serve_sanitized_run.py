"""Calls a serving loop's other entry points of a libsvd build with arguments their host-side
checks reject or only compute sizes from (fake, never dereferenced addresses: no HIP call is
reached), values outside the enumerators and at the ends of the integer types included, and
prints the status codes.  Run by tests/test_abi_serve_sanitized.py."""
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


def attend(c, **kw):
    a = dict(q=4096, qs=256, ctx=64, anc=None, depth=None, off=None, G=0, scale=0.125, cap=0.0,
             slopes=None, B=2, T=3, Hq=4, out=1 << 16, ws=1 << 20, n=0)
    a.update(kw)
    out.append(L.svd_prefix_attention(c, a["q"], a["qs"], a["ctx"], None, a["anc"], a["depth"],
                                      a["off"], a["G"], a["scale"], a["cap"], a["slopes"],
                                      a["B"], a["T"], a["Hq"], a["out"], None, a["ws"], a["n"],
                                      None))


def write_slots(c, **kw):
    a = dict(k=4096, v=8192, dtype=svd.SVD_BF16, ks=128, vs=128, slot=64, N=3)
    a.update(kw)
    out.append(L.svd_cache_write_slots(c, a["k"], a["v"], a["dtype"], a["ks"], a["vs"],
                                       a["slot"], a["N"], None))


BAD = [dict(k=None), dict(dtype=2), dict(dtype=-5), dict(dtype=I32), dict(dtype=-I32 - 1),
       dict(dtype=1), dict(dtype=1, k_scale=65, v_scale=64), dict(head_dim=96),
       dict(head_dim=-I32), dict(page=48), dict(page=-I32 - 1), dict(page=0), dict(n_pages=I64),
       dict(n_pages=-1), dict(kv_heads=I32), dict(kv_heads=-1), dict(k=4100)]
for f in (attend, write_slots):
    f(None)
    for kw in BAD:
        f(cache(**kw))
attend(cache(max_pages=I32))
attend(cache(max_pages=-1))
for kw in (dict(), dict(B=I64), dict(B=1 << 29, T=1), dict(T=I32), dict(T=4096, B=1 << 17),
           dict(Hq=I32), dict(Hq=65536), dict(Hq=-4), dict(scale=3e38), dict(scale=float("nan")),
           dict(scale=1e-45), dict(qs=I64 - 7), dict(qs=-I64), dict(q=4104), dict(out=4096, n=I64),
           dict(ws=(1 << 20) + 8), dict(out=4096 + 512, n=1 << 40), dict(cap=3e38),
           dict(cap=1e-45), dict(cap=-0.0), dict(cap=float("-inf")), dict(off=64, G=I64),
           dict(off=64, G=-I64), dict(off=64, G=2), dict(off=64, G=2, T=4096, B=2),
           dict(off=64, G=1, B=1 << 17, T=4096), dict(slopes=64, depth=64, anc=64)):
    attend(cache(), **kw)
attend(cache(kv_heads=4096, max_pages=(1 << 27) - 1), Hq=65536, B=1 << 17, T=4096, off=64, G=1)
for args in ((1, 1, 32, 8, 128, 4096, 1), (256, 8, 64, 8, 128, 8192, 256), (1, 1, 8, 8, 64, I32, 1),
             (1 << 29, 1, 8, 8, 64, I32, 1 << 29), (1, 4096, 65536, 1, 128, I32, 1),
             (1 << 17, 4096, 65536, 4096, 128, I32, 1 << 17), (I64, 4096, 8, 8, 64, 1, I64),
             (1, 1, 8, 0, 64, 1, 0), (1, 1, 8, 8, 64, I64, 1), (-I64, 1, 8, 8, 64, 1, 0),
             (1, -1, 8, 8, 64, 1, 0), (1, 1, 8, 8, 64, 64, -I64), (1 << 18, 1, 4096, 4096, 64, 64, 1 << 18)):
    out.append(L.svd_prefix_attention_workspace_bytes(*args))
for kw in (dict(dtype=2), dict(dtype=I32), dict(ks=-I64), dict(vs=0), dict(k=4097), dict(N=0),
           dict(N=I64), dict(N=-I64), dict(slot=None)):
    write_slots(cache(block_table=None, max_pages=0), **kw)
for kw in (dict(length=None), dict(B=0), dict(B=I64), dict(B=-I64), dict(B=(1 << 31) - 1, mp=1),
           dict(mp=I32), dict(mp=-I32), dict(page=-I32 - 1), dict(page=I32), dict(n=I64), dict(n=-I64),
           dict(wb=0), dict(so=(1 << 13) + 4), dict(to=(1 << 15) + 4), dict(ws=(1 << 20) + 1)):
    a = dict(length=64, B=4, mp=8, page=16, n=10, ring=1 << 12, state=1 << 13, held=1 << 14,
             table=1 << 15, so=1 << 16, ho=1 << 17, to=1 << 18, room=1 << 19, ws=1 << 20,
             wb=1 << 12)
    a.update(kw)
    out.append(L.svd_cache_pages(a["length"], None, a["B"], a["mp"], a["page"], a["n"], a["ring"],
                                 a["state"], a["held"], a["table"], a["so"], a["ho"], a["to"],
                                 a["room"], a["ws"], a["wb"], None))
for b in (1, 16, 17, 0, I64, -I64, (1 << 31) - 1):
    out.append(L.svd_cache_pages_workspace_bytes(b))
for kw in (dict(c=None), dict(B=0), dict(B=I64), dict(mp=I32), dict(mp=-1), dict(page=I32),
           dict(page=-I32 - 1), dict(n=I64), dict(N=I64), dict(N=-I64)):
    a = dict(c=64, B=4, mp=8, page=16, n=10, N=30)
    a.update(kw)
    out.append(L.svd_cache_slots(a["c"], 128, 256, a["B"], a["mp"], a["page"], a["n"], a["N"], 512,
                                 1024, 2048, 4096, None))
for kw in (dict(z=None), dict(dtype=2), dict(dtype=-I32), dict(B=I64), dict(B=-I64), dict(T=I32),
           dict(V=-I32), dict(z=4097), dict(out=4096 + 2), dict(B=1 << 21, T=2)):
    a = dict(z=4096, out=1 << 20, dtype=svd.SVD_BF16, B=2, T=3, V=100)
    a.update(kw)
    out.append(L.svd_filter_logits(a["z"], a["out"], a["dtype"], a["B"], a["T"], a["V"], None,
                                   None, None, None, None, None))
    if "out" not in kw:
        for K in (1, 65, -I32, I32) if not kw.get("z", 1) else (2,):
            out.append(L.svd_sample(a["z"], a["dtype"], a["B"], a["T"], a["V"], K, None, None,
                                    None, None, None, None, I64, I64, 1 << 20, None, None))
assert svd.SVD_EHIP not in out and svd.SVD_OK not in out[:50], out
print(out)
