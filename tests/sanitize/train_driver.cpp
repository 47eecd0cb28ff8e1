// The operators of include/mps_train.h on the host: every entry point's
// argument checks, with stand-ins for the kernel launchers that count.  A
// refused call must reach no launcher, an accepted one exactly one, with the
// caller's sizes.  Test infrastructure only.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../include/mps_train.h"
#include "../../mixed_precision_sharded_amd/csrc/train_kernels.h"

namespace {
int launches = 0;
int64_t seen_rows = -1, seen_cols = -1;
hipError_t seen(int64_t rows, int64_t cols)
{
    ++launches;
    seen_rows = rows;
    seen_cols = cols;
    return hipSuccess;
}

int failures = 0;
void expect(int line, int rc, int want, const char* word)
{
    static int before = 0;
    const bool launched = launches != before;
    before = launches;
    const bool said = want == 0 || std::strstr(adamw_last_error(), word);
    if (rc != want || launched != (want == 0 && std::strcmp(word, "none") != 0) || !said) {
        std::printf("line %d: rc %d (want %d), launched %d, message '%s'\n", line, rc, want, launched, adamw_last_error());
        ++failures;
    }
}
#define ACCEPT(call) expect(__LINE__, call, 0, "")
#define NOTHING(call) expect(__LINE__, call, 0, "none")
#define REFUSE(call, word) expect(__LINE__, call, MPS_ERR_INVALID_ARGUMENT, word)
#define REFUSE_WS(call, word) expect(__LINE__, call, MPS_ERR_WORKSPACE, word)

constexpr int64_t M = 1 << 20;
char* at(int64_t i) { return reinterpret_cast<char*>(0x7f0000000000) + i * 64 * M; }
uint8_t* bytes(int64_t i) { return reinterpret_cast<uint8_t*>(at(i)); }
float* floats(int64_t i) { return reinterpret_cast<float*>(at(i)); }
constexpr mps_dtype BF = MPS_DTYPE_BF16, F32 = MPS_DTYPE_F32;
const mps_dtype BAD = static_cast<mps_dtype>(7);
}  // namespace

namespace mps {
hipError_t launch_act8_save(Matrix, bool, int64_t r, int64_t c, CodesOut, hipStream_t) { return seen(r, c); }
hipError_t launch_act8_load(Codes, int64_t r, int64_t c, MatrixOut, bool, hipStream_t) { return seen(r, c); }
hipError_t launch_act8_rmsnorm(Matrix, bool, int64_t r, int64_t c, const float*, float, MatrixOut, float*, CodesOut,
                               hipStream_t) { return seen(r, c); }
size_t rmsnorm_backward_scratch(int64_t, int64_t) { return 4096; }
hipError_t launch_act8_rmsnorm_backward(Matrix, bool, Codes, const float*, int64_t r, int64_t c, const float*, Matrix,
                                        MatrixOut, float*, bool, CodesOut, void*, hipStream_t) { return seen(r, c); }
hipError_t launch_act8_swiglu(Matrix, Matrix, bool, int64_t r, int64_t c, MatrixOut, CodesOut, CodesOut, hipStream_t) { return seen(r, c); }
hipError_t launch_act8_swiglu_backward(Matrix, bool, Codes, Codes, int64_t r, int64_t c, MatrixOut, MatrixOut, CodesOut,
                                       hipStream_t) { return seen(r, c); }
size_t weight_grad_scratch(int64_t, int64_t, int64_t) { return 4096; }
hipError_t launch_act8_weight_grad(Matrix, bool, Codes, int64_t t, int64_t, int64_t k, void*, bool, bool, void*, hipStream_t) { return seen(t, k); }
size_t policy_scratch(int64_t, int64_t) { return 4096; }
hipError_t launch_policy_loss(const PolicyArgs& a, bool, void*, hipStream_t) { return seen(a.rows, a.vocab); }
hipError_t launch_zero(float*, int64_t n, hipStream_t) { return seen(0, n); }
}  // namespace mps

int main()
{
    const int64_t big = 1ll << 31;
    // act8_save
    auto save = [](const void* x, mps_dtype t, int64_t stride, int64_t rows, int64_t cols, uint8_t* c, uint8_t* s) {
        return act8_save(x, t, stride, rows, cols, c, s, nullptr);
    };
    ACCEPT(save(at(0), BF, 100, 7, 100, bytes(1), bytes(2)));
    if (seen_rows != 7 || seen_cols != 100) ++failures;
    ACCEPT(save(at(0) + 2, BF, 100, 7, 100, bytes(1), bytes(2) + 1));  // any element-aligned start
    NOTHING(save(nullptr, BF, 100, 0, 100, nullptr, nullptr));
    REFUSE(save(at(0), BAD, 100, 7, 100, bytes(1), bytes(2)), "dtype");
    REFUSE(save(at(0) + 1, BF, 100, 7, 100, bytes(1), bytes(2)), "aligned");
    REFUSE(save(at(0) + 2, F32, 100, 7, 100, bytes(1), bytes(2)), "aligned");
    REFUSE(save(at(0), BF, 100, 7, 100, bytes(1) + 8, bytes(2)), "aligned");
    REFUSE(save(nullptr, BF, 100, 7, 100, bytes(1), bytes(2)), "x is NULL");
    REFUSE(save(at(0), BF, 100, 7, 100, nullptr, bytes(2)), "NULL");
    REFUSE(save(at(0), BF, 100, 7, 100, bytes(1), nullptr), "NULL");
    REFUSE(save(at(0), BF, 99, 7, 100, bytes(1), bytes(2)), "stride");
    REFUSE(save(at(0), BF, 0, 7, 100, bytes(1), bytes(2)), "stride");
    REFUSE(save(at(0), BF, big, 7, 100, bytes(1), bytes(2)), "stride");
    REFUSE(save(at(0), BF, 100, -1, 100, bytes(1), bytes(2)), "rows");
    REFUSE(save(at(0), BF, 100, big, 100, bytes(1), bytes(2)), "rows");
    REFUSE(save(at(0), BF, 100, 7, 0, bytes(1), bytes(2)), "cols");
    REFUSE(save(at(0), BF, big - 1, 7, (1ll << 27) + 1, bytes(1), bytes(2)), "cols");
    REFUSE(save(at(0), BF, 100, 7, 100, bytes(0) + 16, bytes(2)), "overlap");
    REFUSE(save(at(0), BF, 100, 7, 100, bytes(1), bytes(1) + 7 * 128 - 1), "overlap");
    ACCEPT(save(at(0), BF, 100, 7, 100, bytes(1), bytes(1) + 7 * 128));  // one behind the other
    // act8_load
    auto load = [](const uint8_t* c, const uint8_t* s, int64_t rows, int64_t cols, void* x, mps_dtype t, int64_t stride) {
        return act8_load(c, s, rows, cols, x, t, stride, nullptr);
    };
    ACCEPT(load(bytes(0), bytes(1), 3, 33, at(2), F32, 33));
    NOTHING(load(nullptr, nullptr, 0, 33, nullptr, F32, 33));
    REFUSE(load(bytes(0), bytes(1), 3, 33, at(2), BAD, 33), "dtype");
    REFUSE(load(bytes(0), bytes(1), 3, 33, nullptr, F32, 33), "x is NULL");
    REFUSE(load(bytes(0), bytes(1), 3, 33, bytes(0) + 64, F32, 33), "overlap");
    // act8_rmsnorm
    auto norm = [](double eps, void* y, int64_t ys, float* w) {
        return act8_rmsnorm(at(0), BF, 64, 5, 64, w, eps, y, ys, floats(3), bytes(4), bytes(5), nullptr);
    };
    ACCEPT(norm(1e-5, at(1), 64, floats(2)));
    REFUSE(norm(0.0, at(1), 64, floats(2)), "eps");
    REFUSE(norm(-1.0, at(1), 64, floats(2)), "eps");
    REFUSE(norm(1e-60, at(1), 64, floats(2)), "eps");  // 0 in fp32
    REFUSE(norm(1e60, at(1), 64, floats(2)), "eps");
    REFUSE(norm(NAN, at(1), 64, floats(2)), "eps");
    REFUSE(norm(1e-5, at(0), 64, floats(2)), "overlap");  // y over x
    REFUSE(norm(1e-5, at(1), 63, floats(2)), "stride");
    REFUSE(norm(1e-5, at(1), 64, nullptr), "weight");
    REFUSE(norm(1e-5, at(1), 64, floats(3)), "overlap");  // rstd over the weight
    // act8_rmsnorm_backward
    auto back = [](int64_t rows, const void* res, int64_t rs, void* dx, int64_t xs, float* dw, int acc, uint8_t* oc, uint8_t* os,
                   void* ws, size_t wsb) {
        return act8_rmsnorm_backward(at(0), BF, 64, bytes(1), bytes(2), floats(3), rows, 64, floats(4), res, rs, dx, xs, dw, acc,
                                     oc, os, ws, wsb, nullptr);
    };
    ACCEPT(back(5, nullptr, 0, at(5), 64, floats(6), 0, nullptr, nullptr, at(7), 4096));
    ACCEPT(back(5, at(8), 70, at(5), 64, floats(6), 1, bytes(9), bytes(10), at(7), 4096));
    ACCEPT(back(5, at(8), 64, at(8), 64, floats(6), 1, nullptr, nullptr, at(7), 4096));  // dx is the residual's memory
    ACCEPT(back(5, nullptr, 0, at(0), 64, floats(6), 1, nullptr, nullptr, at(7), 4096));  // dx is dy's memory
    REFUSE(back(5, at(8), 64, at(8), 65, floats(6), 1, nullptr, nullptr, at(7), 4096), "overlap");
    REFUSE(back(5, nullptr, 0, at(0) + 2, 64, floats(6), 1, nullptr, nullptr, at(7), 4096), "overlap");
    REFUSE(back(5, nullptr, 0, at(5), 64, floats(4), 0, nullptr, nullptr, at(7), 4096), "overlap");  // dweight over weight
    REFUSE(back(5, nullptr, 0, at(5), 64, floats(6), 0, bytes(9), nullptr, at(7), 4096), "both");
    REFUSE(back(5, nullptr, 0, at(5), 64, floats(6), 0, bytes(1), bytes(10), at(7), 4096), "overlap");
    REFUSE(back(5, at(8), 63, at(5), 64, floats(6), 0, nullptr, nullptr, at(7), 4096), "stride");
    REFUSE(back(5, nullptr, 0, at(5), 64, nullptr, 0, nullptr, nullptr, at(7), 4096), "dweight");
    REFUSE_WS(back(5, nullptr, 0, at(5), 64, floats(6), 0, nullptr, nullptr, nullptr, 4096), "NULL");
    REFUSE_WS(back(5, nullptr, 0, at(5), 64, floats(6), 0, nullptr, nullptr, at(7) + 128, 4096), "aligned");
    REFUSE_WS(back(5, nullptr, 0, at(5), 64, floats(6), 0, nullptr, nullptr, at(7), 4095), "small");
    REFUSE(back(5, nullptr, 0, at(5), 64, floats(6), 0, nullptr, nullptr, at(5) - 3840, 4096), "overlap");
    ACCEPT(back(0, nullptr, 0, nullptr, 64, floats(6), 0, nullptr, nullptr, nullptr, 0));  // zeros
    if (seen_rows != 0 || seen_cols != 64) ++failures;
    NOTHING(back(0, nullptr, 0, nullptr, 64, floats(6), 1, nullptr, nullptr, nullptr, 0));
    REFUSE(back(0, nullptr, 0, nullptr, 64, nullptr, 0, nullptr, nullptr, nullptr, 0), "dweight");
    // act8_swiglu: gate and up as halves of one matrix
    auto gate = [](const void* g, int64_t gs, const void* u, int64_t us, void* o, uint8_t* uc) {
        return act8_swiglu(g, gs, u, us, BF, 6, 40, o, 40, bytes(4), bytes(5), uc, bytes(7), nullptr);
    };
    ACCEPT(gate(at(0), 80, at(0) + 80, 80, at(1), bytes(6)));
    ACCEPT(gate(at(0), 40, at(0), 40, at(1), bytes(6)));  // both inputs the same: only read
    REFUSE(gate(at(0), 80, at(0) + 80, 80, at(0) + 80, bytes(6)), "overlap");
    REFUSE(gate(at(0), 80, at(0) + 80, 80, at(1), bytes(4)), "overlap");
    REFUSE(gate(nullptr, 80, at(0) + 80, 80, at(1), bytes(6)), "gate is NULL");
    REFUSE(gate(at(0), 80, nullptr, 80, at(1), bytes(6)), "up is NULL");
    // act8_swiglu_backward: halves of one matrix written
    auto gback = [](void* dg, int64_t gs, void* du, int64_t us, uint8_t* oc, uint8_t* os) {
        return act8_swiglu_backward(at(0), BF, 40, bytes(1), bytes(2), bytes(3), bytes(4), 6, 40, dg, gs, du, us, oc, os, nullptr);
    };
    ACCEPT(gback(at(5), 80, at(5) + 80, 80, nullptr, nullptr));
    ACCEPT(gback(at(5) + 80, 80, at(5), 80, bytes(6), bytes(7)));
    ACCEPT(gback(at(0), 40, at(5), 40, nullptr, nullptr));  // dgate is dout's memory
    ACCEPT(gback(at(5), 40, at(0), 40, nullptr, nullptr));
    REFUSE(gback(at(0), 40, at(0), 40, nullptr, nullptr), "overlap");
    REFUSE(gback(at(5), 80, at(5) + 78, 80, nullptr, nullptr), "overlap");
    REFUSE(gback(at(5), 80, at(5) + 82, 80, nullptr, nullptr), "overlap");
    REFUSE(gback(at(5), 80, at(5) + 80, 81, nullptr, nullptr), "overlap");
    REFUSE(gback(at(0), 41, at(5), 40, nullptr, nullptr), "overlap");  // dout's memory, another stride
    REFUSE(gback(at(5), 40, at(8), 40, nullptr, bytes(7)), "both");
    REFUSE(gback(at(5), 40, at(8), 40, bytes(1), bytes(7)), "overlap");
    // act8_weight_grad
    auto wgrad = [](int64_t t, int64_t n, int64_t k, int64_t stride, void* dw, mps_dtype dt, int acc, void* ws, size_t wsb) {
        return act8_weight_grad(at(0), BF, stride, bytes(1), bytes(2), t, n, k, dw, dt, acc, ws, wsb, nullptr);
    };
    ACCEPT(wgrad(9, 10, 50, 10, at(3), F32, 0, at(4), 4096));
    ACCEPT(wgrad(9, 10, 50, 10, at(3) + 2, BF, 1, at(4), 4096));
    NOTHING(wgrad(0, 10, 50, 10, at(3), F32, 1, at(4), 4096));
    ACCEPT(wgrad(0, 10, 50, 10, at(3), F32, 0, at(4), 4096));  // zeros
    REFUSE(wgrad(9, 10, 50, 9, at(3), F32, 0, at(4), 4096), "stride");
    REFUSE(wgrad(9, 10, 50, 10, at(3), BAD, 0, at(4), 4096), "dw_dtype");
    REFUSE(wgrad(9, 10, 50, 10, at(3) + 2, F32, 0, at(4), 4096), "aligned");
    REFUSE(wgrad(9, 10, 50, 10, nullptr, F32, 0, at(4), 4096), "dw is NULL");
    REFUSE(wgrad(9, 10, 50, 10, at(0), F32, 0, at(4), 4096), "overlap");
    REFUSE(wgrad(-1, 10, 50, 10, at(3), F32, 0, at(4), 4096), "tokens");
    REFUSE(wgrad(9, 0, 50, 10, at(3), F32, 0, at(4), 4096), "out_features");
    REFUSE(wgrad(9, 10, 0, 10, at(3), F32, 0, at(4), 4096), "in_features");
    REFUSE(wgrad(9, 1 << 27, 1 << 27, 1 << 27, at(3), F32, 0, at(4), 4096), "tiles");
    REFUSE_WS(wgrad(9, 10, 50, 10, at(3), F32, 0, nullptr, 0), "NULL");
    if (act8_weight_grad_workspace_bytes(9, 10, 0) != 0 || !std::strstr(adamw_last_error(), "in_features")) ++failures;
    if (act8_weight_grad_workspace_bytes(9, 10, 5) != 4096 || adamw_last_error()[0]) ++failures;
    if (policy_loss_workspace_bytes(-1, 5) != 0 || !std::strstr(adamw_last_error(), "rows")) ++failures;
    if (act8_rmsnorm_backward_workspace_bytes(0, 5) != 0 || adamw_last_error()[0]) ++failures;
    // policy_loss
    const int64_t* labels = reinterpret_cast<const int64_t*>(at(1));
    auto policy = [&](const float* ref, double lo, double hi, double kl, void* d, int64_t ds, float* loss, float* lp) {
        return policy_loss(at(0), BF, 50, 4, 50, labels, floats(2), ref, floats(3), floats(4), lo, hi, kl, loss, d, ds, lp, nullptr,
                           at(8), 4096, nullptr);
    };
    ACCEPT(policy(floats(5), 0.2, 0.2, 0.1, at(6), 50, floats(7), floats(9)));
    ACCEPT(policy(nullptr, 0.0, 0.0, 0.0, nullptr, 0, floats(7), nullptr));
    ACCEPT(policy(nullptr, 0.2, 0.2, 0.0, at(0), 50, floats(7), nullptr));  // in place
    REFUSE(policy(nullptr, 0.2, 0.2, 0.0, at(0), 51, floats(7), nullptr), "overlap");
    REFUSE(policy(nullptr, 0.2, 0.2, 0.0, at(0) + 2, 50, floats(7), nullptr), "overlap");
    REFUSE(policy(nullptr, 0.2, 0.2, 0.1, at(6), 50, floats(7), nullptr), "ref_logp");
    REFUSE(policy(floats(5), 1.0, 0.2, 0.1, at(6), 50, floats(7), nullptr), "clip_low");
    REFUSE(policy(floats(5), -0.1, 0.2, 0.1, at(6), 50, floats(7), nullptr), "clip_low");
    REFUSE(policy(floats(5), NAN, 0.2, 0.1, at(6), 50, floats(7), nullptr), "clip_low");
    REFUSE(policy(floats(5), 0.2, INFINITY, 0.1, at(6), 50, floats(7), nullptr), "clip_high");
    REFUSE(policy(floats(5), 0.2, -0.2, 0.1, at(6), 50, floats(7), nullptr), "clip_high");
    REFUSE(policy(floats(5), 0.2, 0.2, NAN, at(6), 50, floats(7), nullptr), "kl_coef");
    REFUSE(policy(floats(5), 0.2, 0.2, -1, at(6), 50, floats(7), nullptr), "kl_coef");
    REFUSE(policy(floats(5), 0.2, 0.2, 0.1, at(6), 49, floats(7), nullptr), "stride");
    REFUSE(policy(floats(5), 0.2, 0.2, 0.1, at(6), 50, nullptr, nullptr), "loss is NULL");
    REFUSE(policy(floats(5), 0.2, 0.2, 0.1, at(6), 50, floats(2), nullptr), "overlap");  // loss over old_logp
    REFUSE(policy(floats(5), 0.2, 0.2, 0.1, at(6), 50, floats(7), floats(5)), "overlap");
    ACCEPT(policy_loss(nullptr, BF, 50, 0, 50, nullptr, nullptr, nullptr, nullptr, nullptr, 0.2, 0.2, 0.0, floats(7), nullptr, 0,
                       nullptr, nullptr, nullptr, 0, nullptr));  // no rows: a loss of 0
    REFUSE_WS(policy_loss(at(0), BF, 50, 4, 50, labels, floats(2), nullptr, floats(3), floats(4), 0.2, 0.2, 0.0, floats(7), nullptr,
                          0, nullptr, nullptr, at(8), 100, nullptr), "small");
    // token_logprobs
    auto logp = [&](const int64_t* l, float* out) { return token_logprobs(at(0), F32, 50, 4, 50, l, out, at(8), 4096, nullptr); };
    ACCEPT(logp(labels, floats(2)));
    REFUSE(logp(nullptr, floats(2)), "labels");
    REFUSE(logp(labels, nullptr), "token_logp");
    REFUSE(logp(reinterpret_cast<const int64_t*>(at(1) + 4), floats(2)), "aligned");
    NOTHING(token_logprobs(nullptr, F32, 50, 0, 50, nullptr, nullptr, nullptr, 0, nullptr));
    if (failures) {
        std::printf("%d failures\n", failures);
        return 1;
    }
    std::printf("train driver ok: %d launches\n", launches);
    return 0;
}
