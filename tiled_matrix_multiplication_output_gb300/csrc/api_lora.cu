// C entry points of the low-rank adapters: argument checks, the workspace, and
// the order of the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api_checks.h"
#include "device.h"
#include "grouped_maps.h"
#include "launch.h"
#include "lora.h"
#include "pack.h"
#include "tiled_gemm.h"

using namespace tmmo;

static_assert(kMaxRank == GEMM_MAX_RANK, "the largest rank");

namespace {

size_t round256(int64_t n) { return static_cast<size_t>((n + 255) / 256 * 256); }

// Whether there is an adapter that can change anything.
bool has_adapters(const gemm_lora_t& a) { return a.adapters > 0 && a.rank > 0; }

int check_sizes(const gemm_lora_t* a, int64_t rows, int64_t N, int64_t K, int in_dtype, int out_dtype)
{
    if (!a || !valid_size(rows) || !valid_size(N) || !valid_size(K) || a->adapters < 0 || a->rank < 0 ||
        a->adapters > GEMM_MAX_ADAPTERS || !valid_dtype(in_dtype) || !valid_dtype(out_dtype))
        return GEMM_ERR_INVALID_VALUE;
    return a->rank > GEMM_MAX_RANK ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

int check(const gemm_lora_t* a, const int32_t* adapter, int64_t rows, int64_t N, int64_t K,
          int in_dtype, int out_dtype)
{
    const int rc = check_sizes(a, rows, N, K, in_dtype, out_dtype);
    if (rc != GEMM_OK || !has_adapters(*a))
        return rc;
    if ((rows > 0 && !adapter) || a->stride_a < 0 || a->stride_b < 0)
        return GEMM_ERR_INVALID_VALUE;
    if ((K > 0 && (!a->A || a->lda < K)) || (N > 0 && (!a->B || a->ldb < a->rank)))
        return GEMM_ERR_INVALID_VALUE;
    return GEMM_OK;
}

// The operands as they lie, and the copies that the tensor-core kernels need of
// them (the input X and the output's gradient D: null where a call has none).
struct Operands {
    PackMatrix x, d, w, a, b;
    Packing packing;
    bool tc;  // on the tensor cores; else on the FP32 units, or nothing to sum

    Operands(const void* X, int64_t ldx, const void* D, int64_t ldd, const void* W, int64_t ldw,
             const gemm_lora_t& l, int64_t rows, int64_t N, int64_t K, int in_dtype)
        : x{X, ldx, 0, 1, rows, K}, d{D, ldd, 0, 1, rows, N}, w{W, ldw, 0, 1, N, K},
          a{l.A, l.lda, l.stride_a, l.adapters, l.rank, K},
          b{l.B, l.ldb, l.stride_b, l.adapters, N, l.rank},
          tc(in_dtype != GEMM_F32 && rows > 0 && N > 0 && K > 0)
    {
        if (!tc)
            return;
        for (PackMatrix* m : {&x, &d, &w})
            if (m->p)
                packing.add(m);
        if (has_adapters(l)) {
            packing.add(&a);
            packing.add(&b);
        }
    }
};

// The workspace: `sides` sets of rank values (FP32, or in parts), the plans of
// the row tiles, and the copies.
struct Workspace {
    size_t values, plans, copies;
    int sides;
    // sides 0: the copies alone
    Workspace(int sides_, const gemm_lora_t& l, int64_t rows, int parts, const Operands& o)
        : values(0), plans(0), copies(o.packing.bytes()), sides(sides_)
    {
        if (!has_adapters(l) || sides == 0)
            return;
        values = round256(rows * (o.tc ? lora_parts_bytes(static_cast<int>(l.rank), parts) : l.rank * 4));
        plans = o.tc ? round256((rows + 127) / 128 * LORA_PLAN_BYTES) : 0;
    }
    size_t bytes() const { return sides * values + plans + copies; }
    void* side(void* p, int i) const { return static_cast<char*>(p) + i * values; }
    void* plan(void* p) const { return static_cast<char*>(p) + sides * values; }
    void* copy(void* p) const { return static_cast<char*>(plan(p)) + plans; }
};

// How many parts hold a rank value.  All bits of an FP32 sum in the backward pass, so
// that no gradient depends on the other results' types, and for an FP32 result of BF16
// operands, and for FP16 operands, whose results are finer; two parts are 2^-16 off, a
// 128th of a BF16 result's rounding.
int parts_for(int in_dtype, bool f32_result, bool backward)
{
    return backward || in_dtype == GEMM_F16 || f32_result ? 3 : 2;
}
// How many sets of rank values the backward pass keeps: towards DX and DA, and DB; from FP16
// operands those towards DA are apart (lora_tc.cuh).
int backward_sides(int in_dtype) { return in_dtype == GEMM_F16 ? 3 : 2; }

// Whether one kernel makes the rank values and the product (on the current device).
bool one_kernel(const Operands& o, const gemm_lora_t& l, int64_t rows, int64_t N, int64_t K, int parts)
{
    DeviceInfo d;
    return o.tc && has_adapters(l) && device_info(&d) == cudaSuccess &&
           lora_alone_takes(rows, N, K, l.adapters, static_cast<int>(l.rank), parts, d.num_sms);
}

// The input's direction: rank values from X and A, or (across) from D and B.
LoraLaunch make_launch(const Operands& o, bool across, const gemm_lora_t& lora, const int32_t* adapter,
                       int64_t rows, int64_t N, int64_t K, int in_dtype, const DeviceInfo& d,
                       TensorMaps* maps)
{
    const PackMatrix &in = across ? o.d : o.x, &f = across ? o.b : o.a, &e = across ? o.a : o.b;
    LoraLaunch l{};
    l.X = in.p;
    l.ldx = in.ld;
    l.W = o.w.p;
    l.ldw = o.w.ld;
    l.F = f.p;
    l.ldf = f.ld;
    l.stride_f = f.stride;
    l.E = e.p;
    l.lde = e.ld;
    l.stride_e = e.stride;
    l.across = across;
    l.maps = maps;
    l.scale = lora.scale;
    l.adapter = adapter;
    l.rows = static_cast<int>(rows);
    l.N = static_cast<int>(across ? K : N);
    l.K = static_cast<int>(across ? N : K);
    l.adapters = has_adapters(lora) ? static_cast<int>(lora.adapters) : 0;
    l.rank = static_cast<int>(lora.rank);
    l.in_dtype = in_dtype;
    l.num_sms = d.num_sms;
    l.status = d.status;
    l.wait_budget = wait_budget_cycles();
    l.fault_skip_kblock = fault_skip_kblock();
    return l;
}

}  // namespace

extern "C" size_t gemm_lora_workspace_size(const void* X, int64_t ldx, const void* W, int64_t ldw,
                                           const gemm_lora_t* lora, int64_t rows, int64_t N,
                                           int64_t K, gemm_dtype_t in_dtype, gemm_dtype_t out_dtype)
{
    if (check_sizes(lora, rows, N, K, in_dtype, out_dtype) != GEMM_OK || rows == 0 || N == 0)
        return 0;
    const Operands o(X, ldx, nullptr, 0, W, ldw, *lora, rows, N, K, in_dtype);
    const int parts = parts_for(in_dtype, out_dtype == GEMM_F32, false);
    return Workspace(one_kernel(o, *lora, rows, N, K, parts) ? 0 : 1, *lora, rows, parts, o).bytes();
}

extern "C" int gemm_lora(const void* X, int64_t ldx, const void* W, int64_t ldw,
                         const gemm_lora_t* lora, const int32_t* adapter, void* Y, int64_t ldy,
                         int64_t rows, int64_t N, int64_t K, gemm_dtype_t in_dtype,
                         gemm_dtype_t out_dtype, void* workspace, size_t workspace_bytes,
                         void* stream)
{
    const int rc = check(lora, adapter, rows, N, K, in_dtype, out_dtype);
    if (rc != GEMM_OK || rows == 0 || N == 0)
        return rc;
    if (!Y || ldy < N || (K > 0 && (!X || !W || ldx < K || ldw < K)))
        return GEMM_ERR_INVALID_VALUE;
    Operands o(X, ldx, nullptr, 0, W, ldw, *lora, rows, N, K, in_dtype);
    const int parts = parts_for(in_dtype, out_dtype == GEMM_F32, false);
    const bool alone = one_kernel(o, *lora, rows, N, K, parts);
    const Workspace ws(alone ? 0 : 1, *lora, rows, parts, o);
    if (bad_workspace(workspace, workspace_bytes, ws.bytes()))
        return GEMM_ERR_INVALID_VALUE;
    DeviceInfo d;
    if (device_info(&d) != cudaSuccess)
        return GEMM_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = o.packing.run(ws.copy(workspace), d.num_sms, s);
    TensorMaps maps;
    LoraLaunch l = make_launch(o, false, *lora, adapter, rows, N, K, in_dtype, d, &maps);
    l.Y = Y;
    l.ldy = ldy;
    l.out_dtype = out_dtype;
    l.parts = parts;
    l.t = ws.side(workspace, 0);
    l.plan = ws.plan(workspace);
    if (!o.tc && K == 0)
        l.adapters = 0;
    if (alone)
        return status_of(err == cudaSuccess ? lora_alone_tc_launch(l, s) : err);
    if (err == cudaSuccess && l.adapters > 0)
        err = o.tc ? lora_shrink_tc_launch(l, nullptr, s) : lora_simt_shrink(l, s);
    if (err == cudaSuccess)
        err = o.tc ? lora_expand_tc_launch(l, s) : lora_simt_expand(l, s);
    return status_of(err);
}

extern "C" size_t gemm_lora_backward_workspace_size(const void* D, int64_t ldd, const void* X,
                                                    int64_t ldx, const void* W, int64_t ldw,
                                                    const gemm_lora_t* lora, int64_t rows,
                                                    int64_t N, int64_t K, gemm_dtype_t in_dtype,
                                                    gemm_dtype_t out_dtype,
                                                    gemm_dtype_t grad_dtype)
{
    if (check_sizes(lora, rows, N, K, in_dtype, out_dtype) != GEMM_OK || !valid_dtype(grad_dtype))
        return 0;
    const Operands o(X, ldx, D, ldd, W, ldw, *lora, rows, N, K, in_dtype);
    return Workspace(backward_sides(in_dtype), *lora, rows, parts_for(in_dtype, false, true), o).bytes();
}

extern "C" int gemm_lora_backward(const void* D, int64_t ldd, const void* X, int64_t ldx,
                                  const void* W, int64_t ldw, const gemm_lora_t* lora,
                                  const int32_t* adapter, void* DX, int64_t lddx, void* DA,
                                  int64_t ldda, int64_t stride_da, void* DB, int64_t lddb,
                                  int64_t stride_db, int64_t rows, int64_t N, int64_t K,
                                  gemm_dtype_t in_dtype, gemm_dtype_t out_dtype,
                                  gemm_dtype_t grad_dtype, void* workspace, size_t workspace_bytes,
                                  void* stream)
{
    const int rc = check(lora, adapter, rows, N, K, in_dtype, out_dtype);
    if (rc != GEMM_OK)
        return rc;
    if (!valid_dtype(grad_dtype))
        return GEMM_ERR_INVALID_VALUE;
    const bool adapters = has_adapters(*lora);
    const bool dx = DX && rows > 0 && K > 0;
    const bool da = DA && adapters && K > 0, db = DB && adapters && N > 0;
    if (!dx && !da && !db)
        return GEMM_OK;
    if (rows > 0 && N > 0 && (!D || ldd < N))
        return GEMM_ERR_INVALID_VALUE;
    if ((da || db) && rows > 0 && K > 0 && (!X || ldx < K))
        return GEMM_ERR_INVALID_VALUE;
    if (dx && (lddx < K || (N > 0 && (!W || ldw < K))))
        return GEMM_ERR_INVALID_VALUE;
    if (da && (ldda < K || !apart(lora->adapters, stride_da, lora->rank, ldda, K)))
        return GEMM_ERR_INVALID_VALUE;
    if (db && (lddb < lora->rank || !apart(lora->adapters, stride_db, N, lddb, lora->rank)))
        return GEMM_ERR_INVALID_VALUE;
    Operands o(X, ldx, D, ldd, W, ldw, *lora, rows, N, K, in_dtype);
    const int parts = parts_for(in_dtype, false, true);
    const Workspace ws(backward_sides(in_dtype), *lora, rows, parts, o);
    if (bad_workspace(workspace, workspace_bytes, ws.bytes()))
        return GEMM_ERR_INVALID_VALUE;
    DeviceInfo dev;
    if (device_info(&dev) != cudaSuccess)
        return GEMM_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = o.packing.run(ws.copy(workspace), dev.num_sms, s);

    TensorMaps maps;
    LoraLaunch u = make_launch(o, true, *lora, adapter, rows, N, K, in_dtype, dev, &maps);  // scale * D B
    u.Y = DX;
    u.ldy = lddx;
    u.out_dtype = out_dtype;
    u.parts = parts;
    u.t = ws.side(workspace, 0);
    u.plan = ws.plan(workspace);
    const bool f16 = in_dtype == GEMM_F16;
    if (f16)
        u.t_grad = ws.side(workspace, 2);
    LoraLaunch t = make_launch(o, false, *lora, adapter, rows, N, K, in_dtype, dev, &maps);  // scale * X A^T
    t.parts = parts;
    (f16 ? t.t_grad : t.t) = ws.side(workspace, 1);
    t.plan = u.plan;

    LoraGradLaunch a{};  // dA from X and u
    a.P = o.x.p;
    a.ldp = o.x.ld;
    a.t = f16 ? u.t_grad : u.t;
    a.parts = parts;
    a.plan = u.plan;
    a.maps = &maps;
    a.G = DA;
    a.step_c = 1;
    a.step_j = ldda;
    a.stride_g = stride_da;
    a.adapter = adapter;
    a.rows = u.rows;
    a.cols = static_cast<int>(K);
    a.adapters = u.adapters;
    a.rank = u.rank;
    a.in_dtype = in_dtype;
    a.out_dtype = grad_dtype;
    a.num_sms = u.num_sms;
    a.status = u.status;
    a.wait_budget = u.wait_budget;
    a.fault_skip_kblock = u.fault_skip_kblock;
    LoraGradLaunch b = a;  // dB from D and t
    b.P = o.d.p;
    b.ldp = o.d.ld;
    b.t = f16 ? t.t_grad : t.t;
    b.G = DB;
    b.step_c = lddb;
    b.step_j = 1;
    b.stride_g = stride_db;
    b.cols = static_cast<int>(N);

    auto step = [&](bool wanted, auto launch) {
        if (wanted && err == cudaSuccess)
            err = launch();
    };
    const bool need_u = adapters && (dx || da);
    if (f16 && !dx)
        u.t = nullptr;
    if (f16 && !da)
        u.t_grad = nullptr;
    if (o.tc) {
        step(need_u, [&] { return lora_shrink_tc_launch(u, db ? &t : nullptr, s); });
        step(!need_u && db, [&] { return lora_shrink_tc_launch(t, nullptr, s); });
        step(dx, [&] { return lora_expand_tc_launch(u, s); });
        step(da || db, [&] { return lora_grad_tc_launch({da ? &a : nullptr, db ? &b : nullptr}, dx, s); });
        return status_of(err);
    }
    if (in_dtype != GEMM_F32) {  // sums of nothing: no operand is read
        u.adapters = 0;
        u.K = 0;
        a.rows = b.rows = 0;
    }
    step(u.adapters > 0 && need_u, [&] { return lora_simt_shrink(u, s); });
    step(dx, [&] { return lora_simt_expand(u, s); });
    step(in_dtype == GEMM_F32 && db, [&] { return lora_simt_shrink(t, s); });
    step(da, [&] { return lora_simt_grad(a, s); });
    step(db, [&] { return lora_simt_grad(b, s); });
    return status_of(err);
}
