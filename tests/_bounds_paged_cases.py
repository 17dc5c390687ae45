"""Small ragged cases through the paged-cache entry points, for the bounds-checked build test: run as
    FAQ_LIB=bounds python tests/_bounds_paged_cases.py OUT.npz
(or without FAQ_LIB for the ordinary build); saves every output and exits non-zero if the device
status reports anything.  Inputs are seeded; lengths, groups and pages are off the tile sizes on purpose."""
import os
import sys

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)
import _paged_ref as ref  # noqa: E402
import quantized_attention_amax_b200 as faq  # noqa: E402

# lens, qlens, Hq, Hkv, D, page: single tokens, drafts, blocks of up to 128 rows and of more, empty sequences, long cuts
CASES = [
    ((300, 17, 0, 1000), (1, 1, 1, 1), 16, 4, 128, 64),
    ((257, 31, 64), (4, 0, 5), 6, 2, 64, 32),
    ((513, 90, 5), (40, 90, 9), 4, 4, 64, 16),
    ((1500, 700), (260, 1), 8, 1, 128, 128),
    ((20011, 4097), (3, 40), 8, 2, 128, 1024),
]


def main(path):
    out = {}
    cs = faq.rope_table(21000, 64)
    out["table"] = cs.cpu().numpy()
    for k, (lens, qlens, Hq, H, D, page) in enumerate(CASES):
        for mode in ref.MODES:
            layout = ("BNSD", "BSND")[(k + len(mode)) & 1]
            table, pages = ref.make_table(lens, page, k)
            c = ref.make_cache(mode, layout, pages, H, page, D, 10 + k, spread=0.5)
            cache = faq.PagedCache(c["kc"].cuda(), c["vc"].cuda(), c["ks"].cuda(), c["vs"].cuda(), mode, layout)
            lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
            cu = torch.tensor([0] + list(np.cumsum(qlens)), dtype=torch.int32).cuda()
            batch = faq.PagedBatch(table.cuda(), lens_t, cu)
            T, stride = sum(qlens) + 2, max(lens) + 3
            x = torch.randn((T, Hq + 2 * H, D), generator=torch.Generator().manual_seed(k)).to(torch.bfloat16).cuda()
            amax = [torch.full((H,), 4.0).cuda()] * 2 if mode in ref.PER_HEAD else None
            q, kn, vn = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
            # (sequences with fewer cached tokens than new ones only attend: an append would be reported)
            if all(m <= n for n, m in zip(lens, qlens)):
                q = faq.rope_append(q, kn, vn, cache, batch, cs, interleaved=bool(k & 1), amax=amax, out=torch.zeros_like(q).contiguous())
            else:
                q = q.contiguous()
            res = {"q": q, "o": torch.zeros(T, Hq, D, dtype=torch.bfloat16).cuda(), "lse": torch.zeros(T, Hq).cuda()}
            faq.paged_attention(q, cache, batch, out=res["o"], lse=res["lse"])
            res["o_all"] = faq.paged_attention(q, cache, batch, causal=False, out=torch.zeros_like(res["o"]))
            res["acc"] = faq.paged_weights(q, res["lse"], cache, batch, torch.ones(len(lens), H, stride).cuda())
            res["set"] = faq.paged_weights(q, res["lse"], cache, batch, torch.ones(len(lens), H, stride).cuda(), accumulate=False)
            so = torch.ones_like(res["acc"])
            res["kept"], res["new"] = faq.paged_evict(cache, batch, res["acc"], 50, 3, 7, scores_out=so)
            res.update(so=so, kc=cache.k_codes, vc=cache.v_codes, ks=cache.k_scales, vs=cache.v_scales)
            for name, t in res.items():
                t = t.view(torch.int16) if t.dtype is torch.bfloat16 else t
                out[f"{k}_{mode}_{name}"] = t.cpu().numpy()
            faq.check_device_status()
    np.savez(path, **out)


if __name__ == "__main__":
    main(sys.argv[1])
