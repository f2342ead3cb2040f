// C entry points of the low-rank adapters: argument checks and the
// translation to the internal launchers.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api_checks.h"
#include "device.h"
#include "launch.h"
#include "lora.h"
#include "tiled_gemm.h"

using namespace tmmo;

static_assert(kMaxRank == GEMM_MAX_RANK, "the largest rank");

namespace {

constexpr int64_t kMaxAdapters = 65535;

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

bool valid_sizes(int64_t rows, int64_t N, int64_t K, int64_t adapters, int64_t rank)
{
    return valid_size(rows) && valid_size(N) && valid_size(K) && adapters >= 0 && rank >= 0 &&
           adapters <= kMaxAdapters;
}

// The rank values of all rows: FP32, or in up to three parts.
int64_t values_bytes(int64_t rows, int64_t rank)
{
    return round256(rows * std::max<int64_t>(rank * 4, lora_parts_bytes(static_cast<int>(rank), 3)));
}
int64_t plan_bytes(int64_t rows) { return round256((rows + 127) / 128 * LORA_PLAN_BYTES); }

// How many parts hold a rank value: all bits of an FP32 value for an FP32 result.
int parts_for(int in_dtype, bool f32_result) { return in_dtype == DT_BF16 && f32_result ? 3 : 2; }

// Whether there is an adapter that can change anything.
bool has_adapters(const gemm_lora_t& a) { return a.adapters > 0 && a.rank > 0; }

int check(const gemm_lora_t* a, const int32_t* adapter, int64_t rows, int64_t N, int64_t K,
          int in_dtype, int out_dtype)
{
    if (!a || !valid_sizes(rows, N, K, a->adapters, a->rank) || !valid_dtype(in_dtype) ||
        !valid_dtype(out_dtype))
        return GEMM_ERR_INVALID_VALUE;
    if (a->rank > GEMM_MAX_RANK)
        return GEMM_ERR_UNSUPPORTED;
    if (has_adapters(*a)) {
        if ((rows > 0 && !adapter) || a->stride_a < 0 || a->stride_b < 0)
            return GEMM_ERR_INVALID_VALUE;
        if ((K > 0 && (!a->A || a->lda < K)) || (N > 0 && (!a->B || a->ldb < a->rank)))
            return GEMM_ERR_INVALID_VALUE;
    }
    return GEMM_OK;
}

bool bad_workspace(const void* ws, size_t have, size_t need)
{
    return need > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || have < need);
}

struct Device {
    DeviceInfo info;
    template <typename L>
    void fill(L* l) const
    {
        l->num_sms = info.num_sms;
        l->status = info.status;
        l->wait_budget = wait_budget_cycles();
    }
};

}  // namespace

extern "C" size_t gemm_lora_workspace_size(int64_t rows, int64_t N, int64_t K, int64_t adapters,
                                           int64_t rank)
{
    if (!valid_sizes(rows, N, K, adapters, rank) || rank > GEMM_MAX_RANK)
        return 0;
    return static_cast<size_t>(values_bytes(rows, rank) + plan_bytes(rows));
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
    if (!Y || ldy < N || (K > 0 && (!X || !W || ldx < K || ldw < K)) ||
        bad_workspace(workspace, workspace_bytes,
                      gemm_lora_workspace_size(rows, N, K, lora->adapters, lora->rank)))
        return GEMM_ERR_INVALID_VALUE;
    Device d;
    if (device_info(&d.info) != cudaSuccess)
        return GEMM_ERR_CUDA;
    LoraLaunch l{};
    l.X = X;
    l.ldx = ldx;
    l.W = W;
    l.ldw = ldw;
    l.F = lora->A;
    l.ldf = lora->lda;
    l.stride_f = lora->stride_a;
    l.E = lora->B;
    l.lde = lora->ldb;
    l.stride_e = lora->stride_b;
    l.scale = lora->scale;
    l.adapter = adapter;
    l.Y = Y;
    l.ldy = ldy;
    l.rows = static_cast<int>(rows);
    l.N = static_cast<int>(N);
    l.K = static_cast<int>(K);
    l.adapters = has_adapters(*lora) ? static_cast<int>(lora->adapters) : 0;
    l.rank = static_cast<int>(lora->rank);
    l.in_dtype = in_dtype;
    l.out_dtype = out_dtype;
    l.t = static_cast<float*>(workspace);
    d.fill(&l);
    l.fault_skip_kblock = fault_skip_kblock();
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    l.t16 = workspace;
    l.plan = static_cast<char*>(workspace) + values_bytes(rows, lora->rank);
    l.parts = parts_for(in_dtype, out_dtype == GEMM_F32);
    const bool tc = lora_tc_takes(l);
    cudaError_t err = cudaSuccess;
    if (l.adapters > 0)
        err = tc ? lora_shrink_tc_launch(l, nullptr, s) : lora_simt_shrink(l, s);
    if (err == cudaSuccess)
        err = tc ? lora_expand_tc_launch(l, s) : lora_simt_expand(l, s);
    return status_of(err);
}

extern "C" size_t gemm_lora_backward_workspace_size(int64_t rows, int64_t N, int64_t K,
                                                    int64_t adapters, int64_t rank)
{
    if (!valid_sizes(rows, N, K, adapters, rank) || rank > GEMM_MAX_RANK)
        return 0;
    return static_cast<size_t>(2 * values_bytes(rows, rank) + plan_bytes(rows));
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
    if (da && (ldda < K || (lora->adapters > 1 && !apart(stride_da, lora->rank, ldda, K))))
        return GEMM_ERR_INVALID_VALUE;
    if (db && (lddb < lora->rank || (lora->adapters > 1 && !apart(stride_db, N, lddb, lora->rank))))
        return GEMM_ERR_INVALID_VALUE;
    if (bad_workspace(workspace, workspace_bytes,
                      gemm_lora_backward_workspace_size(rows, N, K, lora->adapters, lora->rank)))
        return GEMM_ERR_INVALID_VALUE;
    Device d;
    if (device_info(&d.info) != cudaSuccess)
        return GEMM_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);

    LoraLaunch l{};  // towards dX: rank values u = scale * D B
    l.X = D;
    l.ldx = ldd;
    l.W = dx ? W : nullptr;
    l.ldw = ldw;
    l.F = lora->B;
    l.ldf = lora->ldb;
    l.stride_f = lora->stride_b;
    l.E = lora->A;
    l.lde = lora->lda;
    l.stride_e = lora->stride_a;
    l.across = true;
    l.scale = lora->scale;
    l.adapter = adapter;
    l.Y = DX;
    l.ldy = lddx;
    l.rows = static_cast<int>(rows);
    l.N = static_cast<int>(K);
    l.K = static_cast<int>(N);
    l.adapters = adapters ? static_cast<int>(lora->adapters) : 0;
    l.rank = static_cast<int>(lora->rank);
    l.in_dtype = in_dtype;
    l.out_dtype = out_dtype;
    l.t = static_cast<float*>(workspace);
    d.fill(&l);
    l.fault_skip_kblock = fault_skip_kblock();

    LoraLaunch f = l;  // forward: rank values t = scale * X A^T
    f.X = X;
    f.ldx = ldx;
    f.F = lora->A;
    f.ldf = lora->lda;
    f.stride_f = lora->stride_a;
    f.across = false;
    f.W = nullptr;
    f.E = lora->B;
    f.lde = lora->ldb;
    f.stride_e = lora->stride_b;
    f.N = static_cast<int>(N);
    f.K = static_cast<int>(K);
    f.t = reinterpret_cast<float*>(static_cast<char*>(workspace) + values_bytes(rows, lora->rank));

    l.t16 = l.t;
    f.t16 = f.t;
    l.plan = f.plan = static_cast<char*>(workspace) + 2 * values_bytes(rows, lora->rank);
    l.parts = f.parts = parts_for(in_dtype, out_dtype == GEMM_F32 || grad_dtype == GEMM_F32);

    LoraGradLaunch a{};  // dA from X and u
    a.P = X;
    a.ldp = ldx;
    a.t = l.t;
    a.t16 = l.t16;
    a.parts = l.parts;
    a.plan = l.plan;
    a.G = DA;
    a.step_c = 1;
    a.step_j = ldda;
    a.stride_g = stride_da;
    a.adapter = adapter;
    a.rows = l.rows;
    a.cols = static_cast<int>(K);
    a.adapters = l.adapters;
    a.rank = l.rank;
    a.in_dtype = in_dtype;
    a.out_dtype = grad_dtype;
    d.fill(&a);
    LoraGradLaunch b = a;  // dB from D and t
    b.P = D;
    b.ldp = ldd;
    b.t = f.t;
    b.t16 = f.t16;
    b.G = DB;
    b.step_c = lddb;
    b.step_j = 1;
    b.stride_g = stride_db;
    b.cols = static_cast<int>(N);

    cudaError_t err = cudaSuccess;
    auto step = [&](bool wanted, auto launch) {
        if (wanted && err == cudaSuccess)
            err = launch();
    };
    const bool need_u = adapters && (dx || da);
    if (rows > 0 && N > 0 && lora_tc_takes(l) && (!adapters || lora_tc_takes(f))) {
        step(need_u || db, [&] {
            return need_u ? lora_shrink_tc_launch(l, db ? &f : nullptr, s) : lora_shrink_tc_launch(f, nullptr, s);
        });
        step(dx, [&] { return lora_expand_tc_launch(l, s); });
        step(da || db, [&] { return lora_grad_tc_launch({da ? &a : nullptr, db ? &b : nullptr}, s); });
        return status_of(err);
    }
    step(need_u, [&] { return lora_simt_shrink(l, s); });
    step(dx, [&] { return lora_simt_expand(l, s); });
    step(db, [&] { return lora_simt_shrink(f, s); });
    step(da, [&] { return lora_simt_grad(a, s); });
    step(db, [&] { return lora_simt_grad(b, s); });
    return status_of(err);
}
