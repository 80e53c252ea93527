"""Gated layers and 8-bit integer products for the device-check build of the library (not collected by
pytest).

``run(gl)`` runs valid launches of each kernel (fp32 of few rows, small tiles, tiles of 256 rows, the
backward's products on either) and returns their outputs and workspace status words as CPU tensors.
``run_tampered(gl)`` runs a backward whose workspace was changed after the offsets call so that the
last group's rows are fewer than none; only the device-check build may run it (dW's tiles of that
group fail their check and are skipped; every access stays inside the buffers either way).

As a script (``python tests/gated_check_cases.py OUT``, with GL_LIBRARY_PATH naming the device-check
build) it runs both and saves the results to OUT with torch.save.
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

DEV = "cuda"
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32

# name: (type, rows of the groups, K, F)
LAYERS = {
    "few": (F32, [3, 0, 5], 260, 68),
    "small": (BF, [5, 0, 40], 264, 72),
    "small_f32": (F32, [70, 0, 33], 132, 516),
    "mid": (F16, [30, 20, 0, 200], 136, 3336),
    "large": (BF, [300, 0, 513], 136, 3464),
    "products": (BF, [130, 0, 400, 257, 300], 2056, 1032),
}
# name: (rows of the groups, K, N)
INT8 = {"int8_small": ([5, 0, 40], 272, 144), "int8_mid": ([30, 20, 0, 200], 272, 6672),
        "int8_large": ([300, 0, 513], 144, 6928)}


def _workspace(gl, m):
    ws = gl.new_workspace(len(m), torch.device(DEV))
    gl.gl_offsets(torch.tensor(m, dtype=torch.int64, device=DEV), int(sum(m)), ws)
    return ws


def run(gl):
    out = {}
    for name, (dt, m, K, F) in LAYERS.items():
        g = torch.Generator().manual_seed(K)
        G, T = len(m), sum(m)
        r = lambda *s: torch.randn(*s, generator=g).to(dt).to(DEV)  # noqa: E731
        new = lambda *s: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
        x, w, b, da, ws = r(T, K), r(G, 2 * F, K) * K ** -0.5, r(G, 2 * F), r(T, F), _workspace(gl, m)
        a, h, dh, dx, dw = new(T, F), new(T, 2 * F), new(T, 2 * F), new(T, K), new(G, 2 * F, K)
        gl.gl_glu_forward(x, w, a, ws, bias=b, h=h)
        gl.gl_glu_backward(x, w, da, dh, dx, dw, ws, bias=b)
        out.update({f"{name}_a": a, f"{name}_h": h, f"{name}_dh": dh, f"{name}_dx": dx, f"{name}_dw": dw,
                    f"{name}_status": torch.tensor(gl.gl_read_status(ws))})
    for name, (m, K, N) in INT8.items():
        g = torch.Generator().manual_seed(K)
        G, T = len(m), sum(m)
        code = lambda *s: torch.randint(-128, 128, s, generator=g, dtype=torch.int8).to(DEV)  # noqa: E731
        x, w, ws = code(T, K), code(G, N, K), _workspace(gl, m)
        xs, wsc = torch.rand(T, generator=g).to(DEV), torch.rand(G, N, generator=g).to(DEV) * 1e-4
        y, a = torch.empty(T, N, dtype=BF, device=DEV), torch.empty(T, N // 2, dtype=BF, device=DEV)
        gl.gl_forward_int8(x, xs, w, wsc, y, ws)
        gl.gl_glu_forward_int8(x, xs, w, wsc, a, ws)
        out.update({f"{name}_y": y, f"{name}_a": a, f"{name}_status": torch.tensor(gl.gl_read_status(ws))})
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in out.items()}


# dW's tiles: of 256 (8 a group) and of 64 (2 a group)
TAMPERED = {"256": (512, 512), "64": (64, 64)}


def run_tampered(gl):
    """16 groups of 16 rows, the last of which ends before it starts: off[16] = 230 < off[15] = 240."""
    out, G = {}, 16
    for name, (K, F) in TAMPERED.items():
        g = torch.Generator().manual_seed(1)
        r = lambda *s: torch.randn(*s, generator=g).to(BF).to(DEV)  # noqa: E731
        x, w, da, h, ws = r(256, K), r(G, 2 * F, K), r(256, F), r(256, 2 * F), _workspace(gl, [16] * G)
        dh = torch.empty(256, 2 * F, dtype=BF, device=DEV)
        ok, dw = (torch.full((G, 2 * F, K), float("nan"), dtype=BF, device=DEV) for _ in range(2))
        gl.gl_glu_backward(x, w, da, dh, None, ok, ws, h=h)
        status_ok = gl.gl_read_status(ws)
        gl.workspace_offsets(ws, G)[G] = 230
        gl.gl_glu_backward(x, w, da, dh, None, dw, ws, h=h)
        out.update({f"tamper_{name}_ok": ok.cpu(), f"tamper_{name}_status_ok": torch.tensor(status_ok),
                    f"tamper_{name}_dw": dw.cpu(), f"tamper_{name}_status": torch.tensor(gl.gl_read_status(ws))})
    torch.cuda.synchronize()
    return out


if __name__ == "__main__":
    import grouped_gemm_gl_amd as gl

    gl.load()
    print(f"gated device-check cases on {gl.library_path}", flush=True)
    res = run(gl)
    print("valid cases done", flush=True)
    res.update(run_tampered(gl))
    print("tampered workspace case done", flush=True)
    res["library"] = torch.tensor(list(gl.library_path.encode()), dtype=torch.uint8)
    torch.save(res, sys.argv[1])
