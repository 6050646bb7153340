"""One fixed set of paged-cache calls, run in its own process against the library NTX_LIB names; outputs, pools, the
bounds-check report and the device status go to an .npz file (argv[1]).  test_gpu_paged_check_build.py runs it once with
the release library and once with the bounds-checked one and compares.

Covered: the cache's write and read of aligned and unaligned rows, unused rows and rows outside the cache, and the
attention of every type, head size and tile width over a narrow table (one launch of clusters) and a wide one (parts and
their join), with empty sequences, lengths past the table and pages outside the pool among them."""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
for p in (ROOT, HERE):
    if p not in sys.path:
        sys.path.insert(0, p)


def main(out_path: str) -> None:
    import numpy as np
    import torch

    import quantized_weight_gemv_dequant_b200 as ntx
    import synthgen as sg

    torch.cuda.init()
    res = {"check_enabled": np.array([ntx.ntx_check_enabled()])}
    ps, lens = 16, [700, 0, 33, 1, 2300, 90]
    used = [-(-n // ps) for n in lens]
    pages = sum(used) + 1
    order = np.random.RandomState(1).permutation(pages)
    statuses = []
    for kind in (ntx.NTX_F16, ntx.NTX_Q8_0, ntx.NTX_Q4_0):
        for d, hkv in ((64, 3), (128, 2), (256, 1)):
            size = ntx.ntx_paged_kv_bytes(kind, hkv, d, ps, pages)
            pools = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
            n, width = sum(lens), hkv * d
            seq = torch.from_numpy(np.repeat(np.arange(6), lens).astype(np.int32)).cuda()
            pos = torch.from_numpy(np.concatenate([np.arange(m) for m in lens]).astype(np.int32)).cuda()
            pos[5] = -1
            seq[6] = 77  # no such sequence
            for positions in (max(used) * ps, 1 << 14):
                table = np.full((6, positions // ps), -1, np.int32)
                i = 0
                for s, u in enumerate(used):
                    table[s, :u] = order[i:i + u]
                    i += u
                tag = f"t{kind}_d{d}_{'narrow' if positions < 8192 else 'wide'}"
                kv = ntx.make_paged_kv(kind, hkv, d, ps, pages, *pools, torch.from_numpy(table).cuda(), 6, positions // ps)
                for pad in (0, 3):
                    stride = width + pad
                    k, v = (torch.from_numpy(sg.fill_f32(2, f"{nm}{tag}{pad}", n * stride)).cuda() for nm in "kv")
                    ntx.ntx_kv_append(kv, k, v, stride, stride, seq, pos, n)
                    back = torch.zeros(2, n, stride, device="cuda")
                    ntx.ntx_kv_read(kv, back[0], back[1], stride, stride, seq, pos, n)
                    res[f"{tag}_read{pad}"] = back.cpu().numpy()
                statuses.append(ntx.ntx_device_status())
                bad = table.copy()
                bad[2, 1] = pages
                kv_bad = ntx.make_paged_kv(kind, hkv, d, ps, pages, *pools, torch.from_numpy(bad).cuda(), 6, positions // ps)
                for group in (1, 4, 7, 16, 40):
                    hq = hkv * group
                    q = torch.from_numpy(sg.fill_f32(3, f"q{tag}{group}", 6 * hq * d)).cuda()
                    ws_n = ntx.ntx_attn_paged_workspace_bytes(kv, hq)
                    ws = torch.full((ws_n,), 0xFF, dtype=torch.uint8, device="cuda")
                    out = torch.full((6, hq, d), float("nan"), device="cuda")
                    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
                    ntx.ntx_attn_decode_paged(kv, q, hq * d, out, hq, ctx, d ** -0.5, ws, ws_n)
                    res[f"{tag}_g{group}"] = out.cpu().numpy()
                    statuses.append(ntx.ntx_device_status())
                    if group == 7:
                        ctx[1], ctx[3] = -3, 2 ** 31 - 1
                        ntx.ntx_attn_decode_paged(kv_bad, q, hq * d, out, hq, ctx, d ** -0.5, ws, ws_n)
                        res[f"{tag}_bad"] = out.cpu().numpy()
                        statuses.append(ntx.ntx_device_status())
            for i in range(2):
                res[f"t{kind}_d{d}_pool{i}"] = pools[i].cpu().numpy()
    res["statuses"] = np.array(statuses)
    site, index = ntx.ntx_check_report()
    res["check_site"] = np.array([site])
    res["check_index"] = np.array([index])
    np.savez(out_path, **res)


if __name__ == "__main__":
    main(sys.argv[1])
